"""64-bit definitions of the 8-bit products with block scales: quantisation, the values that codes and
scales stand for, products grouped by expert."""
from __future__ import annotations

import numpy as np

from . import codecs

BLOCK = 128
MOST = np.float32(448.0)
LEAST = np.float32(2.0 ** -126)


def _scale(top):
    return np.maximum(np.float32(top) / MOST, LEAST)


def quant_rows(x):
    """(codes uint8 [rows, K], scales float32 [rows, KB]) of fp32 values; a NaN is code 0x7F."""
    return _quant(np.asarray(x, np.float32), 1)


def quant_tiles(x):
    """The same with one scale for each tile of 128 rows; x [rows, K]."""
    return _quant(np.asarray(x, np.float32), BLOCK)


def _quant(x, tall):
    rows, K = x.shape
    codes = np.zeros((rows, K), np.uint8)
    scales = np.zeros((-(-rows // tall), -(-K // BLOCK)), np.float32)
    with np.errstate(invalid="ignore", over="ignore"):
        for i in range(scales.shape[0]):
            for j in range(scales.shape[1]):
                part = x[i * tall:(i + 1) * tall, j * BLOCK:(j + 1) * BLOCK]
                mags = np.abs(part)[~np.isnan(part)]
                scales[i, j] = _scale(mags.max() if mags.size else 0.0)
                v = part / scales[i, j]                     # an fp32 quotient
                code = codecs.e4m3_encode_rne_sat(np.where(np.isnan(v), 0.0, v.astype(np.float64)))
                codes[i * tall:(i + 1) * tall, j * BLOCK:(j + 1) * BLOCK] = np.where(np.isnan(v), 0x7F, code)
    return codes, scales


def values(codes, scales, tall=1):
    """What codes [rows, K] stand for."""
    rows, K = codes.shape
    wide = np.repeat(np.repeat(np.asarray(scales, np.float64), tall, axis=0), BLOCK, axis=1)[:rows, :K]
    return codecs.e4m3_decode(codes) * wide


def weight_values(codes, scales, act):
    """What weights [E, N, K] stand for; with act each half of the rows has tiles of its own."""
    E, N, K = codes.shape
    halves = 2 if act else 1
    n, tall = N // halves, scales.shape[1] // halves
    out = np.zeros((E, N, K))
    for e in range(E):
        for h in range(halves):
            out[e, h * n:(h + 1) * n] = values(codes[e, h * n:(h + 1) * n], scales[e, h * tall:(h + 1) * tall], BLOCK)
    return out
