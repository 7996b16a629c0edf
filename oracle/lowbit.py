"""The low-bit operators, written out as plain numpy (TEST INFRASTRUCTURE ONLY).

* AdamW over one tensor with 32-bit states, or with 8-bit moments in blocks
  of 32 with a power-of-two scale;
* the 4-bit wire: blocks of 32 e2m1 codes with a power-of-two scale, chunks of
  a bucket, the coalesced gather's and reduce-scatter's ends.

[codex] 6.3 (the step of a sub-group), 5.2 and 6.2 (what the two collectives
carry) as in ``zero3``; [llmnex] section 3 (what the exchange costs) is why a
narrower wire exists.  The formats are not on the pages: their definition is
the header's, restated here on code tables and binary64 arithmetic.

Pinned by: the published e4m3 type of torch (code table), exhaustive
comparison with all codes (rounding), averages over random words
(stochastic rounding keeps the mean), ``torch.optim.AdamW`` (the update), and
round trips through the 16-bit wire's oracle (places in a chunk).
"""

from __future__ import annotations

from typing import List, Sequence

import numpy as np

from .zero3 import Layout, from_f32, to_f32

BLOCK = 32
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# values of the 8-bit codes: e4m3 magnitudes 0..126 (127 is NaN), and the
# unsigned codes 0..255 with 4 exponent and 4 mantissa bits, both of bias 7
E4M3 = np.array([(m / 8 * 2.0 ** -6) if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])
E4M4 = np.array([(m / 16 * 2.0 ** -6) if e == 0 else (1 + m / 16) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(16)])


# ------------------------------------------------------------ random words

def _mix64(z: int) -> int:
    mask = (1 << 64) - 1
    z ^= z >> 32
    z = z * 0xD6E8FEB86659FD93 & mask
    z ^= z >> 29
    z = z * 0xA0761D6478BD642F & mask
    return z ^ (z >> 32)


def keys(seed: int, step: int, ident: int) -> int:
    mask, g = (1 << 64) - 1, 0x9E3779B97F4A7C15
    return _mix64((_mix64((seed + g * step) & mask) + g * ident) & mask)


def words(key: int, index: np.ndarray) -> np.ndarray:
    """The 32-bit random word of each index, as uint32."""
    i = np.asarray(index, np.uint64)
    k0, k1 = np.uint32(key & 0xFFFFFFFF), np.uint32(key >> 32)
    with np.errstate(over="ignore"):
        x = (i & np.uint64(0xFFFFFFFF)).astype(np.uint32) * np.uint32(0x9E3779B1) + k0
        x = x + (i >> np.uint64(32)).astype(np.uint32) * np.uint32(0x85157AF5)
        x = (x ^ (x >> np.uint32(16))) * np.uint32(0x761BCE4B)
        x = (x ^ (x >> np.uint32(15)) ^ k1) * np.uint32(0xA0D73955)
    return x ^ (x >> np.uint32(16))


# ------------------------------------------------------------------ blocks

def _blocks(x: np.ndarray) -> np.ndarray:
    out = np.zeros(-(-len(x) // BLOCK) * BLOCK, np.float64)
    out[:len(x)] = x
    return out.reshape(-1, BLOCK)


def _scale(top: np.ndarray, fits, lowest: int = -126, highest: int = 127) -> np.ndarray:
    """log2 of the smallest power of two 2^e with fits(top / 2^e), by search from below."""
    e = np.full(top.shape, lowest)
    fin = np.isfinite(top)
    guess = np.where(fin & (top > 0), np.floor(np.log2(np.where(fin & (top > 0), top, 1.0))) - 12, lowest)
    e = np.clip(guess.astype(int), lowest, highest)
    for _ in range(30):
        grow = fin & ~fits(np.ldexp(top, -e)) & (e < highest)
        e = e + grow
    return np.where(fin, e, 128)


def _between(a: np.ndarray, table: np.ndarray):
    """Index of the largest table value <= a, and how far a is to the next, as a fraction."""
    i = np.clip(np.searchsorted(table, a, side="right") - 1, 0, len(table) - 1)
    j = np.minimum(i + 1, len(table) - 1)
    gap = np.where(j > i, table[j] - table[i], 1.0)
    return i, np.where(j > i, (a - table[i]) / gap, 0.0)


# ------------------------------------------------------------ 8-bit moments

def moment_bytes(numel: int) -> int:
    nb = -(-numel // BLOCK)
    return -(-33 * nb // 16) * 16


def encode_moment(x: np.ndarray, word: np.ndarray, second: bool):
    """Codes [numel] and scale bytes of a moment's fp32 values."""
    b = _blocks(np.asarray(x, np.float64))
    bad = ~np.isfinite(b).all(1)
    top = np.where(bad, np.inf, np.abs(np.where(np.isfinite(b), b, 0)).max(1))
    table = E4M4 if second else E4M3
    e = _scale(top, lambda t: t <= table[-1])
    a = np.ldexp(np.abs(np.where(np.isfinite(b), b, 0)), -np.minimum(e, 127)[:, None]).reshape(-1)[:len(x)]
    i, frac = _between(a, table)
    w = word.astype(np.int64)
    if second:      # the word's lower 16 bits; the fraction held to 19 bits
        up = np.rint(frac * 2.0 ** 19).astype(np.int64) + ((w & 0xFFFF) << 3) >= 1 << 19
        code = np.maximum(i + up, np.asarray(x) > 0)
    else:           # its upper 20
        up = np.floor(frac * 2.0 ** 20).astype(np.int64) + (w >> 12) >= 1 << 20
        code = (i + up) | np.where(np.signbit(x), 0x80, 0)
    code = np.where(np.repeat(bad, BLOCK)[:len(x)], 0xFF if second else 0x7F, code)
    return code.astype(np.uint8), np.where(bad, 255, np.clip(e + 127, 1, 254)).astype(np.uint8)


def decode_moment(code: np.ndarray, scale: np.ndarray, second: bool) -> np.ndarray:
    """fp32 values (exact but below fp32's normal range)."""
    c = code.astype(np.int64)
    if second:
        v = E4M4[c]
    else:
        v = np.append(E4M3, np.nan)[c & 0x7F] * np.where(c & 0x80, -1.0, 1.0)
    e = np.repeat(scale.astype(np.int64) - 127, BLOCK)[:len(code)]
    with np.errstate(over="ignore"):
        return np.ldexp(v, e).astype(np.float32)


def moment_buffer(code: np.ndarray, scale: np.ndarray, fill: int = 0) -> np.ndarray:
    nb = len(scale)
    out = np.full(moment_bytes(len(code)), fill, np.uint8)
    out[:len(code)] = code
    out[BLOCK * nb:BLOCK * nb + nb] = scale
    return out


def split_moment(buf: np.ndarray, numel: int):
    nb = -(-numel // BLOCK)
    return buf[:numel], buf[BLOCK * nb:(BLOCK + 1) * nb]


# ------------------------------------------------------------------- AdamW

def adamw(w, m, v, g, *, scale, lr, wd, beta1, beta2, eps, step):
    """One step on fp32 arrays, one fp32 operation each; returns (w, m, v, the
    update's size |lr * ...| in binary64, for error bounds)."""
    f = np.float32
    w, m, v, g = (np.asarray(x, f) for x in (w, m, v, g))
    b1, b2, o1, o2 = f(beta1), f(beta2), f(1.0 - beta1), f(1.0 - beta2)
    with np.errstate(all="ignore"):
        g = g * f(scale)
        if f(lr * wd) != 0:
            w = w - f(lr * wd) * w
        m = b1 * m + o1 * g
        v = b2 * v + o2 * (g * g)
        mh = m / f(1.0 - beta1 ** step)
        vh = v / f(1.0 - beta2 ** step)
        upd = mh / (np.sqrt(vh) + f(eps))
        new = w - f(lr) * upd
        exact = lr * (m.astype(np.float64) / (1 - beta1 ** step)) / (np.sqrt(v.astype(np.float64) / (1 - beta2 ** step)) + eps)
    return new, m, v, w, exact


# ---------------------------------------------------------- the 4-bit wire

def encode4(x: np.ndarray, dtype: str, word=None):
    """Codes (4 bits each, padded to whole blocks) and scale bytes of 16-bit
    values given in fp32; `word`: one random uint32 for each padded element,
    or None for the nearest."""
    b = _blocks(np.asarray(x, np.float64))
    bad = ~np.isfinite(b).all(1)
    top = np.where(bad, np.inf, np.abs(np.where(np.isfinite(b), b, 0)).max(1))
    cap = 13 if dtype == "fp16" else 125
    e = _scale(top, (lambda t: t < 7) if word is None else (lambda t: t <= 6), highest=cap)
    a = np.ldexp(np.abs(np.where(np.isfinite(b), b, 0)), -np.minimum(e, 127)[:, None]).reshape(-1)
    i, frac = _between(np.minimum(a, 6.0), E2M1)
    if word is None:
        up = (frac > 0.5) | ((frac == 0.5) & (i % 2 == 1))
    else:
        up = np.floor(frac * 2.0 ** 32) + word.astype(np.float64) >= 2.0 ** 32
    code = np.minimum(i + up, 7) | np.where(np.signbit(b).reshape(-1), 8, 0)
    code = np.where(np.repeat(bad, BLOCK), 0, code)
    return code.astype(np.uint8), np.where(bad, 255, np.clip(e + 127, 1, 254)).astype(np.uint8)


def decode4(code: np.ndarray, scale: np.ndarray) -> np.ndarray:
    v = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    s = np.repeat(scale.astype(np.int64), BLOCK)
    return np.where(s == 255, np.nan, np.ldexp(v, s - 127)).astype(np.float32)


def bucket_places(layout: Layout, ds_ids: Sequence[int]):
    """(parameters in ascending ds_id, first block of each, blocks of a chunk, chunk bytes)."""
    ps = sorted((layout.slot(int(d)) for d in ds_ids), key=lambda p: p.ds_id)
    nb = [-(-p.partition_size // BLOCK) for p in ps]
    first = np.concatenate([[0], np.cumsum(nb)[:-1]]).astype(int) if ps else np.zeros(0, int)
    blocks = int(sum(nb))
    return ps, first, blocks, -(-17 * blocks // 16) * 16


def _put(chunk: np.ndarray, blocks: int, first: int, code: np.ndarray, scale: np.ndarray) -> None:
    chunk[16 * first:16 * first + len(code) // 2] = code[0::2] | (code[1::2] << 4)
    chunk[16 * blocks + first:16 * blocks + first + len(scale)] = scale


def _get(chunk: np.ndarray, blocks: int, first: int, count: int) -> np.ndarray:
    nb = -(-count // BLOCK)
    b = chunk[16 * first:16 * (first + nb)]
    code = np.stack([b & 15, b >> 4], 1).reshape(-1)
    return decode4(code, chunk[16 * blocks + first:16 * blocks + first + nb])[:count]


def pack4(layout: Layout, rank: int, ds_ids: Sequence[int], shard: np.ndarray, dtype: str, fill: int = 0) -> np.ndarray:
    """The own chunk of a gather bucket (bytes between chunks' ends: `fill`)."""
    ps, first, blocks, size = bucket_places(layout, ds_ids)
    out = np.full(size, fill, np.uint8)
    for p, f in zip(ps, first):
        lo, hi = layout.own_range(p, rank)
        x = np.zeros(p.partition_size, np.float32)
        x[:hi - lo] = to_f32(shard[p.shard_offset:p.shard_offset + hi - lo], dtype)
        _put(out, blocks, f, *encode4(x, dtype))
    return out


def unpack4(layout: Layout, ds_ids: Sequence[int], chunks: Sequence[np.ndarray], dtype: str) -> np.ndarray:
    """The gathered flat buffer (16-bit patterns) from the N chunks."""
    ps, first, blocks, _ = bucket_places(layout, ds_ids)
    out: List[np.ndarray] = []
    for p, f in zip(ps, first):
        full = np.zeros(p.numel, np.uint16)
        for v in range(layout.world_size):
            lo, hi = layout.own_range(p, v)
            if hi > lo:
                full[lo:hi] = from_f32(_get(chunks[v], blocks, f, hi - lo), dtype)
        out.append(full)
    return np.concatenate(out) if out else np.zeros(0, np.uint16)


def send4(layout: Layout, ds_ids: Sequence[int], grads, dtype: str, key=None, fill: int = 0) -> np.ndarray:
    """The send buffer [N, chunk bytes]; grads[ds_id] = 16-bit patterns; `key`:
    of the random words, or None for the nearest."""
    ps, first, blocks, size = bucket_places(layout, ds_ids)
    out = np.full((layout.world_size, size), fill, np.uint8)
    for d in range(layout.world_size):
        for p, f in zip(ps, first):
            lo, hi = layout.own_range(p, d)
            x = np.zeros(-(-p.partition_size // BLOCK) * BLOCK, np.float32)
            x[:hi - lo] = to_f32(grads[p.ds_id][lo:hi], dtype)
            word = None
            if key is not None:
                at = (d * blocks + f) * BLOCK + np.arange(len(x))
                word = words(key, at // 2)
                word = np.where(at % 2 == 0, word, (word << np.uint32(1)) | (word >> np.uint32(31)))
            _put(out[d], blocks, f, *encode4(x, dtype, word))
    return out


def reduce4(layout: Layout, rank: int, ds_ids: Sequence[int], chunks: Sequence[np.ndarray], dtype: str,
            grad_flat: np.ndarray) -> None:
    """The owner's averages, written into grad_flat (16-bit patterns)."""
    ps, first, blocks, _ = bucket_places(layout, ds_ids)
    for p, f in zip(ps, first):
        lo, hi = layout.own_range(p, rank)
        acc = np.zeros(hi - lo, np.float32)
        for v in range(layout.world_size):
            acc = acc + _get(chunks[v], blocks, f, hi - lo)
        out = np.zeros(p.partition_size, np.uint16)
        out[:hi - lo] = from_f32(acc / np.float32(layout.world_size), dtype)
        grad_flat[p.shard_offset:p.shard_offset + p.partition_size] = out
