"""Paged-cache calls on the GPU at their edges: references that move while
other outputs wait."""
import pytest
import torch

import sparse_attention_token_index_b200 as dsa
from paged import DEV, Step, check

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def run(step, out=None, lse=None, **kw):
    kw = {"return_lse": True, "check": True, **step.scale_args(), **kw}
    if out is not None:
        kw.update(out=out, lse=lse)
    if step.idx is None:
        return dsa.dsa_attend_paged(*step.args(), step.max_q, **kw)
    return dsa.dsa_attend_selected(*step.args(), step.idx, **kw)


def loud_tokens(step, loud, jumps):
    """Raises the scores of the positions `loud` (a function of the position) by jumps[h % len] natural units in head h:
    keys and queries get a direction of their own on top of what they hold."""
    u = torch.zeros(step.d, device=DEV)
    u[:16] = 0.25  # |u| = 1
    K = step.K.float()
    K[..., :16] = torch.where(K[..., :16].isnan(), K[..., :16], 0.0)
    for b, n in enumerate(step.lens):
        pos = torch.tensor([p for p in range(n) if loud(p)], device=DEV, dtype=torch.int64)
        if len(pos):
            at = (step.table[b].long()[pos // step.page], pos % step.page)
            K[at[0], at[1]] += 8.0 * u
    step.K.copy_(K.to(step.K.dtype))
    j = torch.tensor([jumps[h % len(jumps)] for h in range(step.Hq)], device=DEV) * step.d ** 0.5 / 8.0
    Q = step.Q.float()
    Q[..., :16] = 0.0
    step.Q.copy_((Q + j[:, None] * u).to(step.Q.dtype))


# ---------------------------------------------------------------------------
# references that move
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("k", [None, 256])
@pytest.mark.parametrize("Hq,m", [(5, 8), (40, 1), (16, 2), (70, 1)])
def test_a_moving_reference_leaves_the_other_outputs(Hq, m, k):
    """Many short caches a multiprocessor, each of two tiles, the second far above the first: every cache's second tile
    scales its own output, while the output of the cache before it still waits to be stored."""
    units = 148 * 3
    if k is None:
        step = Step([256] * units, [m] * units, Hq, 1, 64, page=64, seed=Hq + m)
    else:
        step = Step([300] * (units // m), [m] * (units // m), Hq, 1, 64, page=64, seed=Hq + m, k=k)
        quiet, loud = [p for p in range(256) if p % 2 == 0], [p for p in range(256) if p % 2]
        step.idx.copy_(i32(quiet + loud)[None].expand_as(step.idx))
    loud_tokens(step, (lambda p: p >= 128) if k is None else (lambda p: p % 2 == 1), [20.0, 24.0, 17.0])
    check(step, *run(step))
