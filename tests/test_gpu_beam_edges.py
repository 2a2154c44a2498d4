"""The selection where scores meet the end of their precision: errors of equal terms that add up in lse, logits
whose scores are equal in 64 bits, scores past fp32's range."""

import math

import pytest
import torch

from gated_delta_rule_82_amd import kda
from tests.test_gpu_beam import check

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    kda.load()
    yield
    torch.cuda.synchronize()


def flat(V, dtype, spikes):
    """64 beams (a row is one part then) of `spikes` zeros and V - spikes equal values, -4 to -16: logits, scores
    that make the zeros' continuations about 0, and their distance from it."""
    d = (-4.0 - 12.0 * torch.arange(64) / 63.0).to(dtype)
    x = d.view(1, 64, 1).repeat(1, 1, V).cuda()
    x[:, :, 17:17 + spikes] = 0.0
    lse = [math.log(spikes + (V - spikes) * math.exp(float(y))) for y in d]
    scores = torch.tensor([lse], dtype=torch.float32)
    return x, scores, scores[0].double() - torch.tensor(lse, dtype=torch.float64)


def distances(x, scores, want):
    s, parent, token = kda.beam_select(x, scores.cuda(), 64)
    torch.cuda.synchronize()
    return (s.cpu().double() - want[parent.cpu().long()]).abs(), parent, token


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [32000, 131072, 1 << 20])
def test_a_spike_over_a_flat_row(dtype, V):
    """One large logit and equal ones far below it.  Threads without the spike count ones.  In its own one the spike
    meets five roundings (2^-24) beside the 31 others of its group of loads, and each of the thread's V / 256 or so other
    terms is off by (2 + 1.3 |d|) 2^-24 and meets five too; sums of groups and threads are in 64 bits."""
    x, scores, want = flat(V, dtype, 1)
    far, parent, token = distances(x, scores, want)
    assert sorted(parent[0].tolist()) == list(range(64)) and bool((token == 17).all())
    d = x[0, :, 0].double().cpu()
    tail = (d.exp() * 2.0 ** -24) * (V / 256 + 64) * (7 + 1.3 * d.abs())
    bound = (tail + 5 * 2.0 ** -24 * (1 + 31 * d.exp())) / (1 + (V - 1) * d.exp()) + 1e-10
    assert bool((far[0] <= bound[parent[0].cpu().long()]).all()), (far[0] / bound[parent[0].cpu().long()]).max()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [131072, 1 << 20])
def test_spikes_in_every_thread(dtype, V):
    """Every thread's own terms are far apart: up to 2e-6, as documented."""
    x, scores, want = flat(V, dtype, 2048)
    far, _, _ = distances(x, scores, want)
    assert float(far.max()) <= 2e-6, float(far.max())


@pytest.mark.parametrize("V", [131072, 1 << 20])
@pytest.mark.parametrize("rise", [1e-7, 1e-6, 1e-5])
def test_a_row_that_rises_slowly(V, rise):
    """A new maximum in every group of loads."""
    x = (torch.arange(V, dtype=torch.float64) * rise).float().cuda().view(1, 1, V).repeat(1, 64, 1)
    lse = float(torch.logsumexp(x[0, 0].double(), 0))
    s, _, token = kda.beam_select(x, torch.full((1, 64), lse, device="cuda"), 64)
    torch.cuda.synchronize()
    top = float(x[0, 0, -1].double())
    assert int(token[0, 0]) == V - 1
    assert abs(float(s[0, 0]) - (float(torch.tensor(lse).double()) - lse + top)) <= 2e-6 + 2.0 ** -24 * top


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [300, 20001])
@pytest.mark.parametrize("M", [1, 2, 3, 5, 20])
def test_logits_whose_scores_are_equal(dtype, V, M):
    """Logits so small that 64 bits do not tell their scores apart: within a beam in the order of the logits, whatever
    the number of picks."""
    x = torch.zeros(1, 2, V, dtype=dtype)
    x[0, :, V - 9], x[0, :, 50], x[0, :, 0] = 2e-20, 1e-20, -1e-20
    s, parent, token = kda.beam_select(x.cuda(), torch.tensor([[0.0, -1.0]], device="cuda"), M)
    torch.cuda.synchronize()
    want = [V - 9, 50] + [w for w in range(1, 30) if w != 50]
    assert parent[0].tolist() == [0] * M and token[0].tolist() == want[:M]
    s, parent, token = kda.beam_select(x.cuda(), None, M)       # equal beams: the first one's all come first
    torch.cuda.synchronize()
    assert parent[0].tolist() == [0] * M and token[0].tolist() == want[:M]


def test_scores_past_the_range_of_fp32():
    """A continuation whose score would be rounded to -infinity is none."""
    x = torch.zeros(1, 2, 40)
    x[0, :, 5:] = -2e38
    x[0, 1, 5:9] = -5e37
    s, parent, _ = check(x, torch.tensor([[-3e38, -2.5e38]]), 20)
    assert int((parent >= 0).sum()) == 5 + 5 + 4 and bool(torch.isfinite(s[parent >= 0]).all())
    for dtype in (F32, BF16):       # what the type's lowest value masks, twice
        x = torch.full((1, 1, 40), torch.finfo(dtype).min, dtype=dtype)
        x[0, 0, 3] = 1.0
        s, parent, token = check(x, torch.tensor([[torch.finfo(F32).min]]), 4)
        assert token[0].tolist() == [3, -1, -1, -1]
