"""The KV append names entries that it could not place also where no workspace is given."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import oracle  # noqa: E402
import synth  # noqa: E402
from gpu_helpers import bf16_dev  # noqa: E402

dsa = pytest.importorskip("dsa_indexer_indexshare_gb300")
DEV = torch.device("cuda:0")


def _entries(seq, pos, seed=1):
    x = synth.f32_to_bf16_bits(np.random.default_rng(seed).standard_normal((len(seq), 576)).astype(np.float32))
    t = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    return x, (bf16_dev(x, DEV), t(seq), t(pos))


def _batch():
    return dsa.Batch([0, 1, 2], [199, 49], [0, 200], 256, device=DEV)


@pytest.mark.parametrize("own_stream", [False, True])
@pytest.mark.parametrize("seq,pos", [(2, 3), (-2, 3), (0, -1), (0, 256), (1, 255)])  # the last: beyond the cache
def test_an_entry_outside_raises_and_the_others_are_written(seq, pos, own_stream):
    x, args = _entries([0, seq, 1], [7, pos, 8])
    kv = torch.full((300, 416), 0x5A, dtype=torch.uint8, device=DEV)
    stream, batch = torch.cuda.Stream() if own_stream else None, _batch()
    torch.cuda.synchronize()
    with pytest.raises(dsa.DsaError) as e:
        dsa.dsa_kv_append(*args, batch, kv, stream=stream)
    assert e.value.status == dsa.DSA_ERR_DEVICE_INDEX
    got, want = kv.cpu().numpy(), oracle.kv_int4_quantize(x)
    assert np.array_equal(got[[7, 208]], want[[0, 2]])
    assert (np.delete(got, [7, 208], 0) == 0x5A).all()


def test_padding_and_captured_calls_raise_nothing():
    x, args = _entries([0, -1, 1], [7, 99999, 8])
    kv = torch.zeros((300, 416), dtype=torch.uint8, device=DEV)
    dsa.dsa_kv_append(*args, _batch(), kv)
    want, batch = kv.clone(), _batch()
    kv.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsa.dsa_kv_append(*args, batch, kv)
    assert int(kv.max()) == 0
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(kv, want)
