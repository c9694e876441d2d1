"""Plain 64-bit forms of the 4-bit key/value cache and its attention, and the
documented byte layout of a record, for the tests.

The values a cache holds come from the CPU oracle's quantize_pack (one row per
token and head); the layout functions below are written from the description
in include/qz.h and share nothing with the kernels' index header.
"""
import numpy as np
import torch

import oracle
import synthetic

COMBOS = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 64), (256, 128)]


def bf16_f64(bits):
    return (np.asarray(bits, np.uint32) << 16).view(np.float32).astype(np.float64)


def quantize(x, g):
    """(T, H, D) bf16 tensor -> codes (T, H, D), scales (T, H, D/g) bf16 bits, zeros."""
    T, H, D = x.shape
    if T == 0:
        return (np.zeros((0, H, D), np.uint8), np.zeros((0, H, D // g), np.uint16),
                np.zeros((0, H, D // g), np.uint8))
    c, s, z = oracle.quantize_pack(synthetic.bf16_bits(x.reshape(T * H, D)), 4, False, g)
    codes = np.stack([c & 15, c >> 4], -1).reshape(T, H, D)
    return codes, np.asarray(s).reshape(T, H, D // g), np.asarray(z).reshape(T, H, D // g)


def values(codes, s, z, g):
    """S (q - Z), float64 (exact)."""
    T, H, D = codes.shape
    c = codes.astype(np.float64).reshape(T, H, D // g, g) - z.astype(np.float64)[..., None]
    return (c * bf16_f64(s)[..., None]).reshape(T, H, D)


def record_size(D, g):
    return 16 * D + 96 * (D // g)


def word_byte(word, lane):
    return (word // 4 * 32 + lane) * 16 + word % 4 * 4


def k_place(D, t, d):
    """(byte, high nibble?) of key code d of token t of a record."""
    j, c, n = d // 32, d % 32 // 8, d % 8
    return word_byte(t // 8 * (D // 32) + j, 4 * (t % 8) + c) + n // 2, n % 2


def v_place(D, t, d):
    i, n, e, r = d // 64, d % 64 // 16, d % 16 // 8, d % 8
    return (8 * D + word_byte(t // 8 * (D // 32) + e * (D // 64) + i, 4 * r + t % 8 // 2) +
            2 * (t % 2) + n // 2, n % 2)


def unpack_record(rec, D, g):
    """codes (2, 16, D), scale bits (2, 16, D/g), zeros (2, 16, D/g) of one record's bytes."""
    ng = D // g
    codes = np.empty((2, 16, D), np.uint8)
    for i, place in enumerate((k_place, v_place)):
        for t in range(16):
            for d in range(D):
                byte, high = place(D, t, d)
                codes[i, t, d] = (rec[byte] >> (4 * high)) & 15
    sc = rec[16 * D:16 * D + 64 * ng].view(np.uint16).reshape(2, ng, 16).transpose(0, 2, 1)
    ze = rec[16 * D + 64 * ng:].reshape(2, ng, 16).transpose(0, 2, 1)
    return codes, sc, ze


def attention(q, kv, lens, new, scale, window, masked=None):
    """Per sequence float64 attention.

    q: (T, Hq, D) float64; kv: list of (k^, v^, S_v max per key) per sequence,
    each (len, H, D) float64.  masked[b]: keys to leave out.  Returns out, and
    per output the bound's parts: sum P|v|, sum P S, max P S, |scale| max|q| sum|k|,
    the keys seen, max|v|.
    """
    T, Hq, D = q.shape
    out = np.zeros((T, Hq, D))
    parts = dict(pv=np.zeros((T, Hq, D)), ps=np.zeros((T, Hq, 1)), mps=np.zeros((T, Hq, 1)),
                 dq=np.zeros((T, Hq, 1)), keys=np.zeros((T, Hq, 1)), mv=np.zeros((T, Hq, D)))
    row = 0
    for b, (L, n) in enumerate(zip(lens, new)):
        for i in range(n):
            p = L - n + i
            keep = np.arange(L) <= p
            if window:
                keep &= np.arange(L) > p - window
            if masked is not None:
                keep &= ~masked[b]
            if keep.any():
                k, v, sk, sv = (x[keep] for x in kv[b])
                H = k.shape[1]
                G = Hq // H
                for h in range(Hq):
                    kh, vh = k[:, h // G], v[:, h // G]
                    qh = q[row, h]
                    s = scale * (kh @ qh)
                    e = np.exp(s - s.max())
                    P = e / e.sum()
                    out[row, h] = P @ vh
                    S = sv[:, h // G]
                    parts["pv"][row, h] = P @ np.abs(vh)
                    parts["ps"][row, h] = (P * S).sum()
                    parts["mps"][row, h] = (P * S).max()
                    parts["dq"][row, h] = abs(scale) * np.abs(qh).max() * np.abs(kh).sum(-1).max()
                    parts["keys"][row, h] = keep.sum()
                    parts["mv"][row, h] = np.abs(vh).max(0)
            row += 1
    return out, parts


def bound(out, parts, D):
    """How far the kernel may be from the 64-bit result.

    bf16 result: half a step, 2^-8 of the value.  Weights P S rounded to fp16:
    2^-11 of each, or 2^-25 absolute below its normal range, in units of which
    the largest weight is at least 2^-1 (log2 S is within 2^-20): per key
    15 * 2^-24 of the largest P S.  Scores: a query is held in 16 bits relative
    to its largest value, at most 2^-15 of that off, so a score moves by at most
    |scale| 2^-15 max|q| sum|k|; its integer sum is exact, and the conversion
    and two products round it by less than 2^-21 of |scale| max|q| sum|k|.
    That moves each P by a factor of at most e^(2 delta), and sum |P' - P| |v| by
    no more than 2 max|v| however large delta is (both P sum to 1); ex2 and the
    fp32 sums add 2^-20.  The sum over keys: the tensor core adds 16 products and the
    accumulator with an error of at most 2^-22 of the largest magnitude, sum P S
    15, each time.
    """
    delta = parts["dq"] * (2.0 ** -15 + 2.0 ** -21)
    return (2.0 ** -8 * np.abs(out) +
            ((2.0 ** -11 + 2.0 ** -20) * parts["pv"] +
             np.minimum(np.expm1(np.minimum(2 * delta, 60)) * parts["pv"], 2 * parts["mv"])) *
            (1 + 2.0 ** -8) +
            (parts["keys"] / 16 + 8) * 2.0 ** -22 * 15 * parts["ps"] +
            parts["keys"] * 15 * 2.0 ** -24 * parts["mps"] + 2.0 ** -133)
