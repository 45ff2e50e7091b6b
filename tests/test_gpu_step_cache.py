"""What a captured step leaves in the cache, byte for byte: the keys and values that came out of the projection, the adapters and the
rotation, in the blocks that the plan dealt, by the cache's own definition."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import bit_moe_decode_02_gb300 as moe  # noqa: E402
import test_gpu_kv  # noqa: E402
import test_gpu_kv4  # noqa: E402
from ops_testlib import handle, i32, ok  # noqa: E402
from test_gpu_step import Layer  # noqa: E402


@pytest.mark.parametrize("fmt", [moe.MOE_KV_E4M3, moe.MOE_KV_INT8, moe.MOE_KV_MXFP4])
@pytest.mark.parametrize("D", [64, 128])
def test_the_cache_of_a_captured_step(fmt, D):
    layer, room = Layer(fmt, D=D, seed=4), 60
    layer.buffers(room)
    layer.step()
    ok(handle())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step()
    want = (test_gpu_kv4 if fmt == moe.MOE_KV_MXFP4 else test_gpu_kv).Model(layer.cache)
    lens = [0, 0, 0]
    for counts in ([20, 1, 37], [1, 1, 1], [1, 0, 1], [1, 33, -1], [1, 1, 9], [15, 30, 15], [1, 1, 1]):
        layer.new.copy_(i32(counts))
        layer.x.copy_(torch.randn(layer.x.shape, generator=layer.g, device="cuda"))
        graph.replay()
        ok(handle())
        lens = [0 if n < 0 else a + n for a, n in zip(lens, counts)]
        assert layer.kv_len.tolist() == lens
        layer.cache.table = layer.table.cpu().numpy()
        T = sum(max(n, 0) for n in counts)
        want.write([max(n, 0) for n in counts], lens, layer.k[:T], layer.v[:T])
        want.check()
