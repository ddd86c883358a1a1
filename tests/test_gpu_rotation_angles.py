"""The kernel's cosines, seen through heads whose two products nearly cancel, against
whole-number arithmetic."""
import numpy as np
import pytest
import torch

import angles_ref as A

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def sq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_post_quantized_smooth_amd as sq
    return sq


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,pairs", [(8, 4), (64, 32), (64, 8)])
def test_cosines(sq, D, pairs, interleaved):
    """(a, b) in the ratio of sine to cosine, rounded to fp16: a cos - b sin is their rounding, up
    to 2^-11, and its own rounding to fp16 2^-22 (2^-25 among subnormal numbers). What
    remains: the two errors of cosine and sine, |a|, |b| <= 1, and a product's rounding, 2^-25."""
    rng = np.random.default_rng(D + pairs)
    T = 6000 // pairs
    top = 2.0 ** rng.uniform(0, 31, T)
    top[:T // 4] = 2.0 ** rng.uniform(30, 31, T // 4)
    pos = np.minimum(top, 2 ** 31 - 1).astype(np.int64) * rng.choice([-1, 1], T)
    freq = 1.0 - rng.random(pairs) * 0.4
    freq[0] = 1.0
    x = np.zeros((T, 1, D), np.float16)
    ref, tol = np.zeros((T, pairs)), np.zeros((T, pairs))
    for t in range(T):
        for i in range(pairs):
            c, s = A.exact(pos[t], freq[i])
            n = max(abs(c), abs(s))
            a, b = np.float16(s / n), np.float16(c / n)
            x[t, 0, 2 * i if interleaved else i] = a
            x[t, 0, 2 * i + 1 if interleaved else i + pairs] = b
            ref[t, i] = float(a) * c - float(b) * s
            tol[t, i] = (abs(float(a)) + abs(float(b))) * A.error(pos[t] * freq[i]) + 2.0 ** -25 + \
                abs(ref[t, i]) * 2.0 ** -11 * 1.01 + 2.0 ** -25
    q = torch.from_numpy(x).cuda()
    out = torch.empty_like(q)
    sq.norm_rotary(q, None, out, None, torch.from_numpy(pos.astype(np.int32)).cuda(), torch.from_numpy(freq).cuda(),
                   interleaved=interleaved)
    got = out.cpu().double().numpy()[:, 0]
    got = got[:, 0:2 * pairs:2] if interleaved else got[:, :pairs]
    off = np.abs(got - ref) / tol
    assert off.max() <= 1.0, (off.max(), pos[off.max(1).argmax()])
