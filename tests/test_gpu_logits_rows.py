"""dspark_logits where a work group has several rows of a request: as many
requests and slices of the vocabulary as there is room for.  Cases and bounds
are those of test_gpu_logits."""

import numpy as np
import pytest

from test_gpu_logits import Case, say

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from semi_ar_draft_round_amd import binding
    binding.load_library()
    return torch.device("cuda:0")


# all rows together; several parts of several rows, the first rows only counted; several slices
SIZES = [(2100, 4, 60), (700, 6, 50), (420, 8, 8197), (1030, 1, 2056), (110, 40, 9000)]


@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("R,gamma,V", SIZES)
def test_rows_of_a_work_group(R, gamma, V, dt, packed, dev):
    say(f"[logits] rows {R} {gamma} {V} {dt} {packed}")
    rng = np.random.default_rng(V)
    # few whole requests where rows are long
    ells = [int(x) for x in rng.choice([-1, 0, gamma // 2, gamma - 1, gamma],
                                       R, p=[0.2, 0.2, 0.2, 0.2, 0.2] if V < 1000 else [0.6, 0.1, 0.1, 0.1, 0.1])]
    c = Case(dev, dt, R, gamma, V, ells, packed, seed=R)
    c.nd[: R // 2] = c.nd[: R // 2, :1]                    # one draft all over
    c.check()


@pytest.mark.parametrize("kw", [dict(nb=0, masked=False), dict(history=False, nb=0), dict(history=False, masked=False),
                                dict(drafts=False)])
def test_parts_alone(kw, dev):
    say(f"[logits] rows {kw}")
    for dt in ("f32", "bf16"):
        Case(dev, dt, 2100, 5, 70, [r % 7 - 1 for r in range(2100)], seed=9, **kw).check()
