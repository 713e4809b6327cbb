"""Tensors that a caller gives to the Python binding: shapes, types and places that
the kernels would read or write out of range with are refused before the C call.
The tensors are stand-ins on the host that say they are on a GPU, and the C calls
are replaced by ones that only record that they were reached."""
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")

DEV = torch.device("cuda:0")
NQ, H, K = 5, 16, 8


class OnGpu(torch.Tensor):
    is_cuda = property(lambda t: True)
    device = property(lambda t: DEV)

    def get_device(self):
        return 0


def gpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


@pytest.fixture
def dsa(monkeypatch):
    import dsa_indexer_indexshare_gb300 as m

    reached = []

    class Lib:
        def __getattr__(self, name):
            if name.endswith("workspace_size"):
                return lambda *a: 256
            return lambda *a: reached.append(name) or m.DSA_OK

    fake = Lib()
    monkeypatch.setattr(m, "lib", fake)
    monkeypatch.setattr(m, "_capturing", lambda stream: False, raising=False)
    monkeypatch.setattr(m, "_ATTN", {t: fake.attention for t in m._ATTN})
    return SimpleNamespace(m=m, reached=reached)


def _batch():
    return SimpleNamespace(device=DEV, num_q=NQ, num_seqs=1, max_len=128, c=None, _ref=None)


STREAM = SimpleNamespace(cuda_stream=0)


def _attention(name, dsa, kind="int4", **changed):
    kv = {"bf16": lambda: gpu(64, 576), "fp8": lambda: gpu(64, 656, dtype=torch.uint8),
          "int4": lambda: gpu(64, 416, dtype=torch.uint8)}[kind]()
    a = dict(q_lat=gpu(NQ, H, 512), q_rope=gpu(NQ, H, 64), kv=kv, idx=gpu(NQ, K, dtype=torch.int32),
             out=gpu(NQ, H, 512), lse=gpu(NQ, H, dtype=torch.float32), ws=gpu(4096, dtype=torch.uint8))
    a.update(changed)
    return getattr(dsa.m, name)(a["q_lat"], a["q_rope"], a["kv"], a["idx"], _batch(), scale=1 / 16,
                                out=a["out"], lse=a["lse"], ws=a["ws"], stream=STREAM)


ATTENTION = ["dsa_sparse_mla_attn", "dsa_sparse_mla_attn_rows"]


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("name", ATTENTION)
def test_attention_takes_what_it_needs(dsa, name, kind):
    out, lse = _attention(name, dsa, kind)
    assert out.shape == (NQ, H, 512) and lse.shape == (NQ, H) and len(dsa.reached) == 1
    _attention(name, dsa, kind, idx=gpu(NQ + 3, K, dtype=torch.int32))  # rows behind the batch's are not read
    _attention(name, dsa, kind, lse=gpu(NQ + 3, H, dtype=torch.float32))  # and of a larger buffer not written
    _attention(name, dsa, kind, lse=gpu(NQ * H, dtype=torch.float32))
    assert len(dsa.reached) == 4


@pytest.mark.parametrize("bad", [
    dict(lse=gpu(NQ, H)),                                          # 2 bytes a value
    dict(lse=gpu(NQ - 1, H, dtype=torch.float32)),                 # too short
    dict(lse=gpu(NQ, 2 * H, dtype=torch.float32)[:, ::2]),         # not contiguous
    dict(lse=torch.zeros((NQ, H))),                                # on the host
    dict(ws=torch.zeros(4096, dtype=torch.uint8)),
    dict(ws=gpu(8192, dtype=torch.uint8)[::2]),
    dict(out=gpu(NQ - 1, H, 512)), dict(out=gpu(NQ, H, 512, dtype=torch.float32)),
    dict(out=torch.zeros((NQ, H, 512), dtype=torch.bfloat16)),
    dict(idx=gpu(NQ - 1, K, dtype=torch.int32)),                   # fewer lists than queries
    dict(idx=gpu(NQ * K, dtype=torch.int32)), dict(idx=gpu(NQ, K, dtype=torch.int64)),
    dict(kv=gpu(64, 417, dtype=torch.uint8)),
], ids=lambda d: "-".join(f"{k}_{tuple(v.shape)}_{str(v.dtype)[6:]}_{v.device.type}" for k, v in d.items()))
@pytest.mark.parametrize("name", ATTENTION)
def test_attention_refuses_tensors_it_would_go_beyond(dsa, name, bad):
    with pytest.raises(ValueError):
        _attention(name, dsa, **bad)
    assert not dsa.reached


@pytest.mark.parametrize("name", ATTENTION)
def test_attention_refuses_a_workspace_that_is_none(dsa, name):
    with pytest.raises(TypeError):
        _attention(name, dsa, ws=4096)
    assert not dsa.reached


# ---------------------------------------------------------------- memory of the given stream
I32, F32, U8 = torch.int32, torch.float32, torch.uint8


def _state():
    return SimpleNamespace(c=None, _c=None, num_seqs=1, hot_slots=8, max_pos=128)


def _group():
    return SimpleNamespace(k=K, c=None, num_q=NQ, outs=[], lses=None, layer_types="F", layers=[dict(kv=gpu(64, 576))],
                           workspace_size=lambda batch: 256)


def _hot(m):
    return SimpleNamespace(cold_kv=[gpu(64, 576)], spans=[_state()], rows=gpu(NQ, K, dtype=I32),
                           _c=m._HotGroup())


def _entries():
    return gpu(NQ, dtype=I32), gpu(NQ, dtype=I32)


# every entry point that makes an output or a workspace where the caller gives none
CALLS = {
    "dsa_indexer_scores": lambda m, s, **k: m.dsa_indexer_scores(
        gpu(NQ, 32, 128), gpu(NQ, 32, dtype=F32), gpu(64, 128), _batch(), stream=s, **k),
    "dsa_topk": lambda m, s, **k: m.dsa_topk(gpu(NQ, 128, dtype=F32), _batch(), K, stream=s, **k),
    "dsa_sparse_mla_attn": lambda m, s, **k: m.dsa_sparse_mla_attn(
        gpu(NQ, H, 512), gpu(NQ, H, 64), gpu(64, 576), gpu(NQ, K, dtype=I32), _batch(), scale=1.0, stream=s, **k),
    "dsa_sparse_mla_attn_rows": lambda m, s, **k: m.dsa_sparse_mla_attn_rows(
        gpu(NQ, H, 512), gpu(NQ, H, 64), gpu(64, 576), gpu(NQ, K, dtype=I32), _batch(), scale=1.0, stream=s, **k),
    "dsa_kv_fp8_quantize": lambda m, s, **k: m.dsa_kv_fp8_quantize(gpu(NQ, 576), stream=s, **k),
    "dsa_kv_int4_quantize": lambda m, s, **k: m.dsa_kv_int4_quantize(gpu(NQ, 576), stream=s, **k),
    "dsa_kv_append": lambda m, s, **k: m.dsa_kv_append(gpu(NQ, 576), *_entries(), _batch(), gpu(64, 576), stream=s, **k),
    "dsa_kv_read": lambda m, s, **k: m.dsa_kv_read(gpu(64, 576), *_entries(), _batch(), stream=s, **k),
    "dsa_fp8_quantize": lambda m, s, **k: m.dsa_fp8_quantize(gpu(NQ, 128), stream=s, **k),
    "dsa_indexer_append_keys": lambda m, s, **k: m.dsa_indexer_append_keys(
        gpu(NQ, 128), *_entries(), _batch(), gpu(64, 128), [0.5] * 32, stream=s, **k),
    "dsa_indexer_prepare_queries": lambda m, s, **k: m.dsa_indexer_prepare_queries(
        gpu(NQ, 32, 128), _batch(), [0.5] * 32, fp8=True, stream=s, **k),
    "dsa_hot_plan": lambda m, s, **k: m.dsa_hot_plan(gpu(NQ, K, dtype=I32), _batch(), _state(), 0, stream=s, **k),
    "dsa_hot_fetch": lambda m, s, **k: m.dsa_hot_fetch(_state(), _batch(), [gpu(64, 576)], [gpu(8, 576)], stream=s, **k),
    "indexshare_group_forward": lambda m, s, **k: m.indexshare_group_forward(_group(), _batch(), stream=s, **k),
    "indexshare_group_forward_hot": lambda m, s, **k: m.indexshare_group_forward_hot(
        _group(), _batch(), _hot(m), 0, stream=s, **k),
}


class _TorchThatMakesNothing:
    """torch, whose makers of tensors must not be reached past _made."""

    def __getattr__(self, name):
        if name in ("empty", "zeros", "full"):
            def make(*a, **k):
                raise AssertionError(f"torch.{name} on the current stream")
            return make
        return getattr(torch, name)


@pytest.mark.parametrize("name", CALLS)
def test_a_call_makes_its_tensors_on_the_stream_that_it_works_on(dsa, monkeypatch, name):
    m, made = dsa.m, []
    space = m.workspace

    def record(stream, make, *args, **kw):
        made.append(stream)
        return gpu(4096, dtype=U8) if make is space else gpu(*args[0], dtype=kw["dtype"])

    monkeypatch.setattr(m, "_made", record)
    monkeypatch.setattr(m, "torch", _TorchThatMakesNothing())
    CALLS[name](m, STREAM)
    assert made and all(s is STREAM for s in made) and dsa.reached


def test_every_entry_point_with_a_stream_is_listed(dsa):
    import inspect

    names = {n for n, f in vars(dsa.m).items() if inspect.isfunction(f) and not n.startswith("_")
             and "stream" in inspect.signature(f).parameters}
    # these make nothing: the status of a given workspace, a self-test over one, reads of host pages
    assert names == set(CALLS) | {"status_fetch", "dsa_selftest_wait_timeout", "dsa_hot_touch"}


# ---------------------------------------------------------------- rows that are not written
@pytest.mark.parametrize("given,capturing,fetched", [(False, False, 1), (False, True, 0), (True, False, 0)])
def test_append_without_a_workspace_reports_its_entries(dsa, monkeypatch, given, capturing, fetched):
    m, seen = dsa.m, []
    monkeypatch.setattr(m, "_made", lambda stream, make, *a, **k: gpu(4096, dtype=U8))
    monkeypatch.setattr(m, "_capturing", lambda stream: capturing)
    monkeypatch.setattr(m, "status_fetch", lambda ws, stream=None: seen.append((ws, stream)))
    ws = gpu(4096, dtype=U8) if given else None
    m.dsa_kv_append(gpu(NQ, 576), *_entries(), _batch(), gpu(64, 576), ws=ws, stream=STREAM)
    assert dsa.reached == ["dsa_kv_append"] and len(seen) == fetched
    assert all(s is STREAM for _, s in seen)


# ---------------------------------------------------------------- what the other calls are given
@pytest.mark.parametrize("bad", [lambda: torch.zeros(4096, dtype=U8), lambda: gpu(8192, dtype=U8)[::2]],
                         ids=["on the host", "with gaps"])
@pytest.mark.parametrize("name", sorted(set(CALLS) - {"dsa_kv_fp8_quantize", "dsa_kv_int4_quantize",
                                                      "dsa_fp8_quantize"}))
def test_workspaces_are_checked(dsa, monkeypatch, name, bad):
    made = lambda stream, make, *a, **k: gpu(*a[0], dtype=k["dtype"])  # noqa: E731
    monkeypatch.setattr(dsa.m, "_made", made)
    CALLS[name](dsa.m, STREAM, ws=gpu(4096, dtype=U8))
    reached = list(dsa.reached)
    assert reached
    with pytest.raises(ValueError):
        CALLS[name](dsa.m, STREAM, ws=bad())
    assert dsa.reached == reached


def _raises(dsa, call):
    with pytest.raises(ValueError):
        call()
    assert not dsa.reached


def test_quantiser_outputs_are_checked(dsa):
    x, codes, scale = gpu(NQ, 128), gpu(NQ, 128, dtype=U8), gpu(NQ, dtype=F32)
    dsa.m.dsa_fp8_quantize(x, codes, scale, stream=STREAM)
    dsa.m.dsa_fp8_quantize(x, codes.reshape(-1), scale, stream=STREAM)
    dsa.reached.clear()
    _raises(dsa, lambda: dsa.m.dsa_fp8_quantize(x, codes[1:], scale, stream=STREAM))
    _raises(dsa, lambda: dsa.m.dsa_fp8_quantize(x, codes, scale[1:], stream=STREAM))


def test_key_append_and_query_preparation_are_checked(dsa):
    ws, f = gpu(4096, dtype=U8), [0.5] * 32
    _raises(dsa, lambda: dsa.m.dsa_indexer_append_keys(gpu(NQ, 128), *_entries(), _batch(), gpu(64, 64), f, ws=ws,
                                                       stream=STREAM))
    q, out = gpu(NQ, 32, 128), gpu(NQ, 32, 128, dtype=U8)
    for scale in (gpu(NQ - 1, 32, dtype=F32), gpu(NQ, 32), torch.zeros((NQ, 32))):
        _raises(dsa, lambda: dsa.m.dsa_indexer_prepare_queries(q, _batch(), f, fp8=True, q_out=out, q_scale=scale,
                                                               ws=ws, stream=STREAM))


def test_hot_calls_are_checked(dsa):
    m, ws, small = dsa.m, gpu(4096, dtype=U8), _state()
    small.num_seqs = 0
    rows = gpu(NQ, K, dtype=I32)
    _raises(dsa, lambda: m.dsa_hot_plan(gpu(NQ - 1, K, dtype=I32), _batch(), _state(), 0, rows, ws=ws, stream=STREAM))
    _raises(dsa, lambda: m.dsa_hot_plan(gpu(NQ, K, dtype=I32), _batch(), small, 0, rows, ws=ws, stream=STREAM))
    _raises(dsa, lambda: m.dsa_hot_fetch(small, _batch(), [gpu(64, 576)], [gpu(0, 576)], ws=ws, stream=STREAM))
    hot = _hot(m)
    hot.spans = [small]
    _raises(dsa, lambda: m.indexshare_group_forward_hot(_group(), _batch(), hot, 0, rows, ws=ws, stream=STREAM))
    with pytest.raises(ValueError):
        m.HotGroup([], [gpu(64, 576), gpu(63, 576)], num_q=NQ, k=K, device="cpu")


def test_groups_are_checked(dsa):
    m, ws, few = dsa.m, gpu(4096, dtype=U8), _group()
    few.num_q = NQ - 1
    idx = gpu(NQ, K, dtype=I32)
    _raises(dsa, lambda: m.indexshare_group_forward(few, _batch(), idx, ws=ws, stream=STREAM))
    _raises(dsa, lambda: m.indexshare_group_forward_hot(few, _batch(), _hot(m), 0, idx, ws=ws, stream=STREAM))
    layer = dict(q_lat=gpu(NQ, H, 512), q_rope=gpu(NQ, H, 64), kv=gpu(64, 576), q_idx=gpu(NQ, 32, 128, dtype=U8),
                 w=gpu(NQ, 32, dtype=F32), k_idx=gpu(64, 128, dtype=U8), q_scale=gpu(NQ, 32, dtype=F32),
                 k_scale=gpu(64, dtype=F32))
    make = lambda out, **k: m.Group("F", [dict(layer, **k)], k=K, scale=1.0, outs=out)  # noqa: E731
    make([gpu(NQ, H, 512)])
    make([gpu(NQ + 2, H, 512)])
    for out in ([gpu(NQ - 1, H, 512)], [gpu(NQ, H, 512, dtype=F32)], [torch.zeros((NQ, H, 512), dtype=torch.bfloat16)], []):
        with pytest.raises(ValueError):
            make(out)
    with pytest.raises(ValueError):
        make([gpu(NQ, H, 512)], k_scale=gpu(63, dtype=F32))


def test_a_batch_on_the_host_has_no_device_number(dsa):
    assert dsa.m.Batch([0, 1], [0], [0], 128, device=torch.device("cpu", 0)).device.index is None
