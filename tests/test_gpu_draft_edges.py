"""The drafter's calls at the edges of what their documentation allows: lists without entries,
log-sum-exps that do not belong to their list, temperatures near the smallest number, several host
threads, outputs left out. Tolerances stand beside each test."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import draft_token_verification_spec_b200 as sv
from tests import _draft_ref as ref
from tests.test_gpu_distill import check, teacher
from tests.test_gpu_sample import check_sample, check_top, make, uniforms

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


# ------------------------------------------------------------------------- distillation
@pytest.mark.parametrize("rows", [6, 200])
@pytest.mark.parametrize("V,dtype", [(3000, F32), (40000, BF16), (150000, F32)])
def test_a_list_without_entries_costs_nothing(V, dtype, rows):
    """Exactly nothing, in one call as in two, whatever the row's log-sum-exp is."""
    if V == 150000:
        rows = min(rows, 20)
    x = make(rows, V, dtype)
    ids, val, lse = teacher(x, 12, short=False)
    ids[:rows // 2] = -1
    val[rows // 2:] = -math.inf
    for l in (None, lse):
        loss, _ = sv.spec_distill_loss(x, ids, val, l)
        both_loss, grad = sv.spec_distill_loss_grad(x, ids, val, l)
        assert (loss == 0.0).all() and (both_loss == 0.0).all() and (grad == 0.0).all()
    x[1, 5] = math.nan               # still a row in error
    loss, grad = sv.spec_distill_loss_grad(x, ids, val, lse)
    assert torch.isnan(loss[1]) and torch.isnan(grad[1].float()).all() and (loss[2:] == 0.0).all()
