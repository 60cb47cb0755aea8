"""The example's speculative decoding, step by step against a plain model: the
cache holds the committed text's keys and values in order, and every
committed token is the one that the plain model's processed logits choose
(where their two largest are further apart than bf16 attention moves them)."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import serving_ref as ref

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "speculative_step.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("speculative_step", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_commits_what_the_plain_model_chooses(example):
    model, cache, _, text, lens, prompt, processors, kept = example.run(B=4, V=499, steps=6,
                                                                        depth=3)
    assert (kept >= 0).all() and int((kept > 0).sum()) > 0 and int((kept < 3).sum()) > 0
    assert torch.equal(lens, prompt + (kept + 1).sum(0).to(torch.int32))
    assert torch.equal(cache.len, lens - 1)
    host = {k: (v.cpu().numpy().view(np.uint32) if k == "mask_words" else v.cpu().numpy())
            for k, v in processors.items()}
    checked = 0
    for b in range(4):
        n, first = int(lens[b]), int(prompt[b])
        tokens = text[b:b + 1, :n]
        x, q, k, v = model.project(tokens, torch.arange(n, device="cuda")[None])
        at = torch.arange(n - 1, device="cuda")
        blocks = cache.table[b, at // cache.page].long()
        # the projections of another batch shape: fp32 sums that round to bf16 one step apart at most
        for c, want in ((cache.k, k), (cache.v, v)):
            got, want = c[blocks, at % cache.page].float(), want[0, :n - 1].float()
            assert ((got - want).abs() <= 2.0 ** -7 * want.abs() + 2.0 ** -12).all()

        table = np.zeros((1, 1), np.int32)
        mask = None
        for i in range(first, n):                  # token i, chosen after the first i
            out, _, weight, _ = ref.attention(
                q[:, i - 1:i].double().cpu().numpy(), k[:, :i].double().cpu().numpy(),
                v[:, :i].double().cpu().numpy(), table, [i - 1], [1], mask, model.dim ** -0.5)
            a = torch.from_numpy(out).cuda()
            raw = (x[0, i - 1].double() + model.mix * a.flatten()) @ model.head.double()
            y, _ = ref.logits(raw.cpu().numpy()[None, None], text[b:b + 1].cpu().numpy(),
                              [first], [i], None, None, host["repetition"][b:], host["frequency"][b:],
                              None, host["bias_ids"][b:], host["bias_values"][b:], None,
                              host["mask_words"], np.zeros((1, 1), np.int64))
            # what two roundings to bf16 of each attention element can move a difference of logits by
            moved = model.mix * 2.0 ** -8 * (torch.from_numpy(2 * np.abs(out) + weight).cuda().flatten()
                                     @ model.head.double().abs()).max()
            top = np.sort(y[0, 0])[-2:]
            if top[1] - top[0] > 2 * float(moved):
                assert int(y[0, 0].argmax()) == int(text[b, i])
                checked += 1
    assert checked > 10
