"""What a call returns: tensors of their own, which may be resized, freed, saved or written without the others."""
import io

import pytest
import torch

import memory_bound_elementwise_gb300 as ew
from tests.rows_util import randn

pytestmark = pytest.mark.gpu


def calls():
    logits, one = randn((6, 40), 1), randn((6,), 2)
    tokens = torch.arange(6, device="cuda")
    x, w = randn((6, 64), 3), randn((64,), 4)
    experts = (torch.arange(12, device="cuda") % 5).view(6, 2)
    y, h, mean, rstd = ew.ew_layernorm(x, w, w, residual=x)
    return {"sort": ew.ew_expert_sort(experts, 5, align=4), "policy": ew.ew_policy(logits, tokens, one),
            "policy step": ew.ew_policy_step(logits, tokens, one, one), "layer norm": (y, h, mean, rstd),
            "its gradient": ew.ew_layernorm_grad(x, h, w, mean, rstd), "norm": ew.ew_rmsnorm(x, w, residual=x),
            "log probabilities": ew.ew_logprob(logits, tokens, top=2),
            "distillation": ew.ew_distill(logits, tokens[:, None], one[:, None])}


def test_outputs_share_no_storage():
    for name, outs in calls().items():
        places = [t.untyped_storage().data_ptr() for t in outs]
        assert len(set(places)) == len(outs), name
        for t in outs:
            assert t.storage_offset() == 0 and t.untyped_storage().nbytes() == t.numel() * t.element_size(), name


def test_a_resized_output_leaves_the_others_alone():
    for name, outs in calls().items():
        before = [t.clone() for t in outs]
        for k, t in enumerate(outs):
            t.resize_(t.numel() * 16).fill_(7)
            for other, want in zip(outs[k + 1:], before[k + 1:]):
                assert torch.equal(other, want), name


def test_a_saved_output_is_no_larger_than_itself():
    n = 4096
    loss, logp, lse = ew.ew_policy(randn((n, 8), 5), torch.zeros(n, dtype=torch.int64, device="cuda"), randn((n,), 6))
    for t in (loss, logp, lse):
        with io.BytesIO() as f:
            torch.save(t.cpu(), f)
            least = f.tell()
        with io.BytesIO() as f:
            torch.save(t, f)
            assert f.tell() < least + 4 * n
