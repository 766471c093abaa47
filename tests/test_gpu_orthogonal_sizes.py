"""Orthogonalised updates where the product with N takes several runs of
columns to a workgroup, at ranks past 256, and at the ends of float32.

Tolerances are oracle.orthogonal.tolerance, for the coefficients and eps that
the call takes, which are float32.  (Given the decimals in 64 bits instead, the
oracle's own result moves by up to 5.83 of that tolerance in the first case of
test_ranks_past_256, adapter 1, by the coefficients' rounding of 2^-25 alone:
they enter elements of Q where c1 G and c2 G^2 nearly cancel.)"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from lora_adapter_amd import binding as B
from oracle import orthogonal as NS
from tests.test_gpu_orthogonal import COEF, EPS, Fleet, run_ortho, step_once

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()


def compare(fl, v, out, ads, steps=5, eps=EPS):
    coef, eps = [float(np.float32(c)) for c in COEF], float(np.float32(eps))
    for a in ads:
        N = v[fl.rows(a)].astype(np.float64)
        off = np.abs(out[fl.rows(a)] - NS.newton_schulz(N, steps, coef, eps))
        tol = NS.tolerance(N, steps, coef, eps) + 2.0 ** -149
        assert np.all(off <= tol), (a, float(np.max(off / tol)))


@pytest.mark.parametrize("M", [4200, 6200])
def test_several_runs_of_columns(M):
    """832 columns are four runs of 256, the last of 64; with 4 M runs over
    16384 a workgroup takes two of them (M = 4200), or three and then one."""
    ranks = np.random.default_rng(M).integers(1, 3, size=M).tolist()
    fl = Fleet(ranks, 832, 64, seed=M)
    v = fl.values(832)
    out, ork = run_ortho(fl, torch.from_numpy(v).cuda(), list(range(M)), 2)
    assert ork == ranks
    compare(fl, v, out, range(M))
    spare = np.ones(fl.n_pages, bool)
    spare[fl.ids] = False
    assert (out[spare] == 7).all()


def test_several_runs_of_columns_over_rank_128():
    """Ranks over 128 stage Q and the pages again for every run."""
    ranks = np.random.default_rng(3).integers(1, 4, size=1500).tolist()
    for a, r in ((0, 130), (7, 128), (700, 129), (1300, 66), (1499, 130)):
        ranks[a] = r
    fl = Fleet(ranks, 832, 64, seed=12)
    v = fl.values(832)
    out, ork = run_ortho(fl, torch.from_numpy(v).cuda(), list(range(1500)), 130)
    assert ork == ranks
    compare(fl, v, out, [a for a in range(1500) if ranks[a] > 3 or a % 50 == 1])


@pytest.mark.parametrize("ranks,d,steps", [([300, 5], 832, 3), ([257, 256], 320, 2), ([1024], 1088, 2)])
def test_ranks_past_256(ranks, d, steps):
    fl = Fleet(ranks, d, d, seed=sum(ranks))
    v = fl.values(d)
    out, ork = run_ortho(fl, torch.from_numpy(v).cuda(), list(range(len(ranks))), max(ranks), steps)
    assert ork == ranks
    compare(fl, v, out, range(len(ranks)), steps)


def test_subnormal_rows():
    ranks = [1, 2, 3, 3, 5, 16, 70, 40]
    fl = Fleet(ranks, 1088, 64, seed=31)
    v = (fl.values(1088).astype(np.float64) * 2.0 ** -130).astype(np.float32)
    out, _ = run_ortho(fl, torch.from_numpy(v).cuda(), list(range(len(ranks))), 70, eps=1e-20)
    compare(fl, v, out, range(len(ranks)), eps=1e-20)


@pytest.mark.parametrize("nesterov", [None, False, True])
def test_norms_past_2_to_the_126(nesterov):
    """.. whose reciprocal is no normal float32: rows of numbers up to 1e38,
    orthogonalised, and as the gradient of a step."""
    ranks = [1, 3, 16, 33, 70]
    fl = Fleet(ranks, 4160, 4160, seed=17)
    v = fl.rng.uniform(-1e38, 1e38, (fl.n_pages, 4160)).astype(np.float32)
    ads = list(range(len(ranks)))
    if nesterov is None:
        out, _ = run_ortho(fl, torch.from_numpy(v).cuda(), ads, 70)
        compare(fl, v, out, ads)
        return
    # a step of lr 1 on pages of zero with no decay leaves -O; momentum 0 makes N the gradient
    zero = lambda: torch.zeros(fl.n_pages, 4160, device="cuda")
    fl.pages = [zero(), zero()]
    grad = torch.from_numpy(v).cuda()
    keep = step_once(fl, ads, 70, [zero(), zero()], [grad, grad], [None, None], (1.0, 1.0), 0.0, nesterov, 0.0)
    torch.cuda.synchronize()
    for p in fl.pages:
        compare(fl, v, -p.double().cpu().numpy(), ads)
