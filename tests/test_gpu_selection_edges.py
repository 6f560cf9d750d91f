"""Calls of the selection operators at the ends of their ranges, on the GPU
against the plain 64-bit implementation.  Tolerances are those of
test_gpu_route.py and test_gpu_logits.py, which state how they are made."""
import numpy as np
import pytest

from test_gpu_route import check_route

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


# -------------------------------------------------- scores near binary64's end

@pytest.mark.parametrize("E,G,kept", [(16, 1, 1), (16, 4, 3), (300, 1, 1), (1024, 8, 4),
                                      (512, 512, 500), (1000, 200, 150)])
def test_sigmoid_scores_near_the_end_of_binary64(E, G, kept):
    """Scores of 1e-300 to 1e-308 differ in binary64, and from -709.78 down
    they are 0: the choice under a bias is theirs, whichever kernel makes it
    (the last two shapes are those of the kernel that is binary64 throughout)."""
    rng = np.random.default_rng([E, G])
    z = np.linspace(-708.5, -690.5, E)[None].repeat(6, 0)
    z[1] = z[0][::-1]
    z[2] = rng.permutation(z[0])
    z[3, : E // 2] = -720.0
    z[4] = np.where(rng.random(E) < 0.8, -750.0, z[2])
    z[5] = rng.choice([-700.0, -705.0, -691.0], size=E)
    z = z.astype(np.float32)
    for bias in (np.zeros(E, np.float32), np.full(E, 2.0 ** -149, np.float32)):
        check_route(torch.from_numpy(z), z, score="sigmoid", top_k=5, groups=G, kept_groups=kept,
                    group_top=1, bias=bias)
