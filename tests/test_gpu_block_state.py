"""What an attention block keeps between calls: its cache after a refused call."""
import pytest
import torch

from test_gpu_block import make, tokens

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def sq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_post_quantized_smooth_amd as sq
    return sq


def test_a_retry_after_a_refused_call_is_the_call(sq):
    B, K, Hq, Hkv, D = 2, 256, 4, 2, 64
    block, _ = make(sq, K, Hq, Hkv, D)
    X = tokens(B, 12, K, torch.float16)
    caches = [sq.KeyValueCache(B, 16, Hkv, D, torch.float16) for _ in range(2)]
    for c in caches:
        block(X[:, :9], cache=c)
    for kw in (dict(causal=False, prefix=torch.zeros(B, dtype=torch.int32, device="cuda")),
               dict(key_ranges=torch.zeros(B + 1, 3, 2, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            block(X[:, 9:], cache=caches[1], **kw)
    want, got = (block(X[:, 9:], cache=c)[0] for c in caches)
    assert torch.equal(want, got) and caches[0].length == caches[1].length == 12
    assert torch.equal(caches[0].k[:, :12], caches[1].k[:, :12])
