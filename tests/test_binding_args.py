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


@pytest.mark.parametrize("bad", [
    dict(lse=gpu(NQ, H)),                                          # 2 bytes a value
    dict(lse=gpu(NQ - 1, H, dtype=torch.float32)),                 # too short
    dict(lse=gpu(NQ * H, dtype=torch.float32)),
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
