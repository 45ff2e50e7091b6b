"""The example's decode loop: the operators and the expert block together."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import bit_moe_decode_02_gb300 as moe  # noqa: E402
from bit_moe_decode_02_gb300 import build_ext  # noqa: E402
from examples.decode import Model  # noqa: E402


@pytest.mark.parametrize("fmt", [moe.MOE_KV_E4M3, moe.MOE_KV_INT8])
def test_generates_and_repeats(fmt):
    build_ext.build()
    prompts = [[1, 2, 3], [4] * 90, [5]]
    runs = []
    for _ in range(2):
        model = Model(streams=3, cache_format=fmt)
        runs.append(model.generate(prompts, 6))
        assert model.lengths == [3 + 5, 90 + 5, 1 + 5]
        model.close()
    assert runs[0] == runs[1]
    assert all(len(t) == 6 and all(0 <= x < 1000 for x in t) for t in runs[0])


def test_prompt_at_once_and_token_by_token():
    """The same 70 tokens in one call and in 70: the cache's codes differ only where a block's scale grew on the way, and
    the batched expert path quantises its activations; the last token's logits stay close."""
    build_ext.build()
    tokens = [(11 * i) % 1000 for i in range(70)]
    at_once, one_by_one = Model(streams=1), Model(streams=1)
    a = at_once.forward([tokens])[0][-1].double()
    for t in tokens:
        b = one_by_one.forward([[t]])[0][-1]
    b = b.double()
    assert torch.corrcoef(torch.stack((a, b)))[0, 1] > 0.9
    at_once.close()
    one_by_one.close()
