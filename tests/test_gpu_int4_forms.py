"""Every form of the attention over INT4 rows that the dispatch chooses from: 16, 32 and
64 heads, lists of at most half a block and longer ones, a token split over 1 to 16
CTAs, contiguous and paged caches and absolute rows.  The outputs are equal bit for
bit to the bf16 attention on the values the rows stand for (32 heads, which that does
not take: to the first half of 64 heads over the same rows), and the same whatever the
cache's layout."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import oracle  # noqa: E402
import synth  # noqa: E402
from gpu_helpers import bf16_dev, make_batch  # noqa: E402
from test_gpu_kvint4 import T, _attention_inputs, _check_oracle, _vs_bf16  # noqa: E402

dsa = pytest.importorskip("dsa_indexer_indexshare_gb300")
DEV = torch.device("cuda:0")
SCALE = 1 / 16
LENS = [2600, 130, 2500, 3000]
# queries of each sequence: splits of 16, 8, 4, 2 and 1 at K = 2048, of 4 to 1 at K = 500
QUERIES = {1: [1, 0, 0, 0], 7: [2, 1, 3, 1], 25: [10, 1, 9, 5], 50: [40, 2, 5, 3], 170: [130, 30, 9, 1]}


def _paged(lay, kv4, R, seed):
    """The same cache in blocks of R rows in random order; rows of no position are NaN."""
    nb = [(n + R - 1) // R for n in LENS]
    ids = np.random.default_rng(seed).permutation(sum(nb) + 1)
    table = np.full((len(LENS), (lay.max_len + R - 1) // R), -1, np.int32)
    phys = np.full(((sum(nb) + 1) * R, 416), 0xFF, np.uint8)
    for b, n in enumerate(LENS):
        table[b, :nb[b]] = ids[sum(nb[:b]):sum(nb[:b + 1])]
        s = np.arange(n)
        phys[table[b, s // R].astype(np.int64) * R + s % R] = kv4[lay.seq_row0[b] + s]
    batch = dsa.Batch(lay.q_start, lay.q_pos, None, lay.max_len, device=DEV, block_table=table, block_rows=R)
    return batch, phys, table


@pytest.mark.parametrize("H", [16, 32, 64])
@pytest.mark.parametrize("K,queries", [(33, 7), (33, 170), (64, 25), (64, 170), (65, 50), (500, 1), (500, 7), (500, 50),
                                       (500, 170), (2048, 1), (2048, 7), (2048, 25), (2048, 50), (2048, 170)])
def test_every_form_gives_the_same_bits(H, K, queries):
    lay, ql, qr, kv4, idx = _attention_inputs(LENS, QUERIES[queries], H, K, seed=H + K + queries, holes=K % 2 == 1)
    Q, R_, I = bf16_dev(ql, DEV), bf16_dev(qr, DEV), T(idx)
    deq = oracle.kv_int4_dequantize(kv4)
    want, wl = _vs_bf16(Q, R_, kv4, deq, idx, make_batch(dsa, lay, DEV), SCALE)
    _check_oracle(want, wl, lay, ql, qr, deq, idx, SCALE, np.unique(np.linspace(0, lay.num_q - 1, 5).astype(int)))
    R = 128 if (K + queries) % 2 else 512
    paged, phys, table = _paged(lay, kv4, R, seed=K)
    ws = dsa.workspace(dsa.lib.dsa_sparse_mla_workspace_size(paged.c, H, K), DEV)
    out, lse = dsa.dsa_sparse_mla_attn(Q, R_, T(phys), I, paged, scale=SCALE, ws=ws)
    assert dsa.status_fetch(ws) == 0
    assert torch.equal(out, want) and torch.equal(lse, wl)
    seq = np.searchsorted(lay.q_start, np.arange(lay.num_q), side="right") - 1
    pos = np.maximum(idx, 0)
    rows = np.where(idx >= 0, table[seq[:, None], pos // R].astype(np.int64) * R + pos % R, -1).astype(np.int32)
    out, lse = dsa.dsa_sparse_mla_attn_rows(Q, R_, T(phys), T(rows), paged, scale=SCALE, ws=ws)
    assert dsa.status_fetch(ws) == 0
    assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("H", [16, 32, 64])
@pytest.mark.parametrize("K", [64, 300])
def test_many_tokens_of_unequal_weight_on_one_cta(H, K):
    """More than 128 tokens' worth of work items a CTA: lists of many tokens, some of
    which see one position, some K, some nothing at all."""
    lens, qc = [5000, 40, 700], [4900, 40, 1]
    lay, ql, qr, kv4, idx = _attention_inputs(lens, qc, H, K, seed=H + K)
    rng = np.random.default_rng(K)
    idx[rng.random(lay.num_q) < 0.2] = -1
    few = rng.random(lay.num_q) < 0.3
    idx[few, 1:] = -1
    Q, R_ = bf16_dev(ql, DEV), bf16_dev(qr, DEV)
    out, lse = _vs_bf16(Q, R_, kv4, oracle.kv_int4_dequantize(kv4), idx, make_batch(dsa, lay, DEV), SCALE)
    empty = T((idx < 0).all(1))
    assert (out[empty] == 0).all() and torch.isneginf(lse[empty]).all()
    assert torch.isfinite(lse[~empty]).all()
