"""Calls on a stream that is not the current one: what they make for themselves is
of that stream's memory, so the current stream is not given it while they run."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import oracle  # noqa: E402
import synth  # noqa: E402
from gpu_helpers import bf16_dev, device_layers, make_batch  # noqa: E402

dsa = pytest.importorskip("dsa_indexer_indexshare_gb300")
DEV = torch.device("cuda:0")
LENS = [900, 2000, 1500]


def _behind_a_delay(nbytes, call):
    """call(stream) behind a delay on its stream, while the current stream takes and
    fills memory of the sizes that the call needs."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)
    got = call(s)
    mine = [torch.zeros(n, dtype=torch.uint8, device=DEV) for n in nbytes for _ in range(3)]
    torch.cuda.synchronize()
    assert all((m == 0).all() for m in mine)
    return got


@pytest.mark.parametrize("kind", ["bf16", "int4"])
def test_attention_over_absolute_rows(kind):
    lay = synth.make_layout(LENS, [1, 1, 1])
    rng = np.random.default_rng(1)
    g = lambda *s: synth.f32_to_bf16_bits(rng.standard_normal(s).astype(np.float32))  # noqa: E731
    kv = bf16_dev(g(lay.rows, 576), DEV)
    kv = dsa.dsa_kv_int4_quantize(kv) if kind == "int4" else kv
    q, r = bf16_dev(g(3, 64, 512), DEV), bf16_dev(g(3, 64, 64), DEV)
    rows = torch.from_numpy(np.stack([lay.seq_row0[b] + rng.permutation(n)[:800] for b, n in enumerate(LENS)])
                            .astype(np.int32)).to(DEV)
    batch = make_batch(dsa, lay, DEV)
    want, wl = dsa.dsa_sparse_mla_attn_rows(q, r, kv, rows, batch, scale=1 / 16)
    n = dsa.lib.dsa_sparse_mla_workspace_size(batch.c, 64, 800)
    out, lse = _behind_a_delay([n, want.numel() * 2], lambda s: dsa.dsa_sparse_mla_attn_rows(
        q, r, kv, rows, batch, scale=1 / 16, stream=s))
    assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("kind", ["bf16", "int4"])
def test_group_calls(kind):
    types, K, slots = "FSFS", 128, 300
    lay = synth.make_layout(LENS, [1, 1, 1])
    batch = make_batch(dsa, lay, DEV)
    layers = device_layers(synth.host_layers(lay, types, 64, ints=False, seed=2), DEV)
    for L in layers:
        L["kv"] = dsa.dsa_kv_int4_quantize(L["kv"]) if kind == "int4" else L["kv"]
    group = dsa.Group(types, layers, k=K, scale=1 / 16)
    outs, _, widx = dsa.indexshare_group_forward(group, batch)
    want = [o.clone() for o in outs]
    sizes = [group.workspace_size(batch), 3 * K * 4]
    outs, _, idx = _behind_a_delay(sizes, lambda s: dsa.indexshare_group_forward(group, batch, stream=s))
    assert torch.equal(idx, widx) and all(torch.equal(a, b) for a, b in zip(outs, want))

    cold = [L["kv"].cpu().pin_memory() for L in layers]
    hot_layers = [dict(L, kv=torch.zeros((3 * slots, L["kv"].shape[1]), dtype=L["kv"].dtype, device=DEV))
                  for L in layers]
    hgroup = dsa.Group(types, hot_layers, k=K, scale=1 / 16)
    hot = dsa.HotGroup([dsa.HotState(3, slots, lay.max_len, DEV) for _ in range(2)], cold, num_q=3, k=K,
                       device=DEV)
    outs, _, idx = _behind_a_delay(sizes, lambda s: dsa.indexshare_group_forward_hot(
        hgroup, batch, hot, 0, stream=s))
    assert torch.equal(idx, widx) and all(torch.equal(a, b) for a, b in zip(outs, want))


def test_indexer_topk_and_cache_calls():
    """Scores, selection, query preparation and the key append, one after the other on
    the stream, each making its own output."""
    lay = synth.make_layout(LENS, [1, 1, 1])
    batch = make_batch(dsa, lay, DEV)
    L = device_layers(synth.host_layers(lay, "F", 16, ints=False, seed=3), DEV)[0]
    freq = oracle.rope_inv_freq(8e6)
    seq = torch.arange(3, dtype=torch.int32, device=DEV)
    pos = torch.tensor(LENS, dtype=torch.int32, device=DEV) - 1
    new = L["k_idx"][:3].clone()

    def step(s=None):
        keys = L["k_idx"].clone() if s is None else keys_s
        dsa.dsa_indexer_append_keys(new, seq, pos, batch, keys, freq, stream=s)
        q = dsa.dsa_indexer_prepare_queries(L["q_idx"], batch, freq, stream=s)
        scores = dsa.dsa_indexer_scores(q, L["w"], keys, batch, stream=s)
        return q, scores, dsa.dsa_topk(scores, batch, 64, stream=s)

    want = step()
    keys_s = L["k_idx"].clone()
    sizes = [want[1].numel() * 4, want[0].numel() * 2, dsa.lib.dsa_topk_workspace_size(batch.c, 64),
             dsa.lib.dsa_indexer_workspace_size(batch.c)]
    got = _behind_a_delay(sizes, step)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
