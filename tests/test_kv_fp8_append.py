"""FP8 rows have one definition, whichever call writes them: the scale is the fp32
nearest to amax / 448 and a code the E4M3 value nearest to the exact x / scale."""
from fractions import Fraction as F

import numpy as np
import pytest

import oracle
import synth


def _rows(n, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, 576)) * np.exp2(rng.integers(-20, 20, (n, 1)))
    b = synth.f32_to_bf16_bits(x.astype(np.float32))
    if n > 8:
        b[1, :512] = 0            # zero groups: scale 1
        b[2, :512] = 0x8000
        b[3, 5] = 0x7F7F          # the largest finite value
        b[4, :512] = 0
        b[4, 0:512:128] = [1, 3, 77, 0x0080]  # subnormals and the smallest normal value
    return b


def _scales(rows):
    return np.ascontiguousarray(rows[:, 512:528]).view(np.float32)


def test_append_rows_are_the_quantisers():
    b = _rows(400, 1)
    a = oracle.kv_append_rows(b, np.zeros(400, np.int32), None, "fp8")
    assert np.array_equal(a, oracle.kv_fp8_quantize(b))
    # the fp32 nearest to the exact quotient: no nearer neighbour
    amax = np.abs(synth.bf16_bits_to_f32(b[:, :512])).reshape(400, 4, 128).max(axis=2)
    for s, m in list(zip(_scales(a).ravel(), amax.ravel()))[:800]:
        if m == 0:
            assert s == 1
            continue
        want, far = F(float(m)) / 448, abs(F(float(s)) - F(float(m)) / 448)
        assert all(far <= abs(F(float(np.nextafter(s, t))) - want)
                   for t in (np.float32(0), np.float32(np.inf)))


@pytest.mark.gpu
@pytest.mark.parametrize("paged", [False, True])
def test_gpu_append_equals_the_quantiser_bit_for_bit(paged):
    """The same rows by both calls: finite rows of every size, equal bytes; NaN and
    infinities, equal values."""
    torch = pytest.importorskip("torch")
    dsa = pytest.importorskip("dsa_indexer_indexshare_gb300")
    from gpu_helpers import bf16_dev

    dev, n, R = torch.device("cuda:0"), 4000, 128
    b = _rows(n, 2)
    b[10, 7], b[11, 130], b[12, 300], b[13, 511] = 0x7FC0, 0x7F80, 0xFF80, 0xFFC1
    x = bf16_dev(b, dev)
    nb = (n + R - 1) // R
    table = np.random.default_rng(3).permutation(nb).astype(np.int32)[None]
    batch = (dsa.Batch([0, 1], [n - 1], None, nb * R, device=dev, block_table=table, block_rows=R) if paged
             else dsa.Batch([0, 1], [n - 1], [0], nb * R, device=dev))
    seq = torch.zeros(n, dtype=torch.int32, device=dev)
    pos = torch.arange(n, dtype=torch.int32, device=dev)
    kv = torch.zeros((nb * R, 656), dtype=torch.uint8, device=dev)
    ws = dsa.workspace(256, dev)
    dsa.dsa_kv_append(x, seq, pos, batch, kv, ws=ws)
    assert dsa.status_fetch(ws) == 0
    p = np.arange(n)
    rows = table[0, p // R].astype(np.int64) * R + p % R if paged else p
    got = kv[torch.from_numpy(rows).to(dev)].cpu().numpy()
    want = dsa.dsa_kv_fp8_quantize(x).cpu().numpy()
    fin = np.ones(n, bool)
    fin[10:14] = False
    assert np.array_equal(got[fin], want[fin])
    assert np.array_equal(got[fin], oracle.kv_fp8_quantize(b[fin]))
    val = lambda r: synth.bf16_bits_to_f32(oracle.kv_fp8_dequantize(r))  # noqa: E731
    assert np.array_equal(val(got[10:14]), val(want[10:14]), equal_nan=True)
