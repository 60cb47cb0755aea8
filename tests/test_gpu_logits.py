"""dspark_logits_process against the definition in 64 bits.  Each of the at
most five steps (scale, count times frequency, two subtractions, each bias)
is one fp32 rounding of a value below the sum of the terms' magnitudes, so
the result is within (4 + biases) 2^-24 of that sum, then within half a
step of the type; untouched logits come through bit for bit."""
import math

import numpy as np
import pytest
import torch

import draft_sampling_verification_gb300 as ds
import serving_ref as ref

pytestmark = pytest.mark.gpu

U = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8}


class Case:
    def __init__(self, B, rows, V, dtype=torch.float32, history=50, drafts=None, biases=0, masks=0,
                 tree=False, seed=0):
        rng = np.random.default_rng(seed)
        self.x = torch.from_numpy(rng.normal(0, 4, (B, rows, V)).astype(np.float32)).to(dtype)
        ids = lambda *s: (V ** rng.random(s)).astype(np.int32) - 1  # noqa: E731
        nd = rows - 1 if drafts is None else drafts
        self.kw = dict(history=None, prompt_len=None, history_len=None, draft_tokens=None,
                       row_mask=None, repetition=(1 + rng.random(B)).astype(np.float32),
                       frequency=rng.random(B).astype(np.float32),
                       presence=rng.random(B).astype(np.float32), bias_ids=None, bias_values=None,
                       n_bias=None, mask_words=None, mask_rows=None)
        k = self.kw
        if history:
            k["history"] = ids(B, history)
            k["history"][:, ::7] = rng.integers(-3, V + 3, k["history"][:, ::7].shape)
            k["history_len"] = rng.integers(0, history + 1, B).astype(np.int32)
            k["prompt_len"] = (k["history_len"] * rng.random(B)).astype(np.int32)
        if nd:
            k["draft_tokens"] = ids(B, nd)
            if history and nd > 1:
                k["draft_tokens"][:, 1] = k["history"][:, 0]
            if nd > 2:
                k["draft_tokens"][:, 2] = k["draft_tokens"][:, 0]
                k["draft_tokens"][0, 1] = -1
        if tree:
            k["row_mask"] = rng.integers(0, 1 << 63, (B, rows), dtype=np.uint64)
        if biases:
            k["bias_ids"] = rng.integers(0, V, (B, biases)).astype(np.int32)
            k["bias_ids"][:, -1] = k["bias_ids"][:, 0]
            k["bias_values"] = rng.normal(0, 3, (B, biases)).astype(np.float32)
            k["n_bias"] = rng.integers(0, biases + 1, B).astype(np.int32)
            k["n_bias"][0] = biases
        if masks:
            k["mask_words"] = rng.integers(0, 1 << 32, (masks, (V + 31) // 32)).astype(np.uint32)
            k["mask_rows"] = rng.integers(-1, masks, (B, rows)).astype(np.int32)

    def device(self):
        d = {}
        for n, t in self.kw.items():
            if t is not None and t.dtype in (np.uint64, np.uint32):
                t = t.view(np.int64 if t.dtype == np.uint64 else np.int32)
            d[n] = None if t is None else torch.from_numpy(t).cuda()
        return d

    def run(self, x=None, **kw):
        x = self.x.cuda() if x is None else x
        r = ds.logits_process(x, **self.device(), **kw)
        torch.cuda.synchronize()
        return r

    def check(self, out):
        k = self.kw
        x = self.x.double().numpy()
        want, size = ref.logits(x, k["history"], k["prompt_len"], k["history_len"],
                                k["draft_tokens"], k["row_mask"], k["repetition"], k["frequency"],
                                k["presence"], k["bias_ids"], k["bias_values"], k["n_bias"],
                                k["mask_words"], k["mask_rows"])
        got = out.double().cpu().numpy()
        n = 4 + (0 if k["bias_ids"] is None else k["bias_ids"].shape[1])
        fine = np.isfinite(want)
        tol = n * 2.0 ** -24 * size * (1 + U[self.x.dtype]) + U[self.x.dtype] * np.abs(
            np.where(fine, want, 0))
        assert np.array_equal(got[~fine], want[~fine], equal_nan=True)
        assert (np.abs(got[fine] - want[fine]) <= tol[fine]).all()
        same = (want == x) & fine                # untouched: bit for bit
        assert (got[same] == x[same]).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 7, 31, 257, 1000, 4096, 4099, 20011])
@pytest.mark.parametrize("rows", [1, 6])
def test_everything_at_once(dtype, V, rows):
    c = Case(3, rows, V, dtype, history=90, biases=min(V, 20), masks=4, seed=V + rows)
    out, status = c.run()
    c.check(out)
    assert (status == 0).all()


@pytest.mark.parametrize("what", [dict(history=0), dict(drafts=0), dict(biases=700),
                                  dict(masks=1), dict(tree=True), dict(history=3000),
                                  dict(history=1), dict(tree=True, drafts=64, masks=2)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_parts(what, dtype):
    c = Case(4, 6, 5003, dtype, seed=3, **what)
    c.check(c.run()[0])


@pytest.mark.parametrize("missing", [["repetition"], ["frequency"], ["presence"],
                                     ["prompt_len"], ["n_bias"], ["mask_rows"],
                                     ["repetition", "frequency", "presence"]])
def test_optional_arguments(missing):
    c = Case(2, 3, 777, biases=9, masks=6, seed=4)
    for m in missing:
        c.kw[m] = None
    c.check(c.run()[0])


def test_sixty_four_rows_and_a_full_vocabulary():
    c = Case(1, 64, 3001, torch.bfloat16, drafts=63, tree=True, masks=64, history=400)
    c.check(c.run()[0])
    c = Case(2, 2, 131072, torch.bfloat16, history=2000, biases=100, masks=2)
    c.check(c.run()[0])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("masks", [0, 3])
def test_in_place(dtype, masks):
    c = Case(3, 6, 4099, dtype, biases=30, masks=masks, seed=6)
    want, _ = c.run()
    x = c.x.cuda()
    out, _ = c.run(x, out=x)
    assert out is x and torch.equal(x, want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("ld,shift,ld_out,shift_out", [(4099, 0, 4099, 0), (4104, 1, 4104, 1),
                                                       (5000, 3, 4200, 0), (4101, 2, 4107, 5)])
def test_strides_and_alignment(dtype, ld, shift, ld_out, shift_out):
    """Rows at any element: source and destination may sit differently within 16 bytes."""
    c = Case(2, 3, 4099, dtype, biases=5, masks=3, seed=7)
    want, _ = c.run()

    def rows(width, at):
        flat = torch.full((6 * width + at + 16,), 5.0, dtype=dtype, device="cuda")
        return flat, flat[at:at + 6 * width].view(2, 3, width)[..., :4099]

    _, x = rows(ld, shift)
    x.copy_(c.x)
    flat, y = rows(ld_out, shift_out)
    c.run(x, out=y)
    assert torch.equal(y, want)
    y.fill_(5.0)                                 # nothing outside the rows was written
    assert (flat == 5.0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_extreme_logits(dtype):
    """Infinities, NaN and the type's lowest value: through the steps like any number, and gone
    under a mask."""
    c = Case(1, 2, 64, dtype, history=0, drafts=0, masks=1)
    c.x[0, :, :8] = torch.tensor([math.nan, math.inf, -math.inf, torch.finfo(dtype).min,
                                  torch.finfo(dtype).max, 0.0, -0.0, 1.0])
    k = c.kw
    k["history"] = np.arange(6, dtype=np.int32)[None]
    k["history_len"], k["prompt_len"] = np.array([6], np.int32), np.array([2], np.int32)
    k["repetition"] = np.array([2.0], np.float32)
    k["mask_words"] = np.array([[0xFFFFFF00, 0xFFFFFFFF]], np.uint32)
    k["mask_rows"] = np.array([[0, -1]], np.int32)
    out, _ = c.run()
    out = out.float().cpu()
    assert torch.isneginf(out[0, 0, :8]).all() and torch.isfinite(out[0, 0, 8:]).all()
    assert math.isnan(out[0, 1, 0]) and out[0, 1, 1] == math.inf and out[0, 1, 2] == -math.inf
    assert out[0, 1, 3] == -math.inf             # lowest value times 2
    assert math.isfinite(out[0, 1, 4]) and out[0, 1, 7] == 1.0


def test_all_masked_row_is_refused_by_the_verifier():
    c = Case(1, 2, 100, history=0, masks=1)
    c.kw["mask_words"][:] = 0
    c.kw["mask_rows"] = np.zeros((1, 2), np.int32)
    out, _ = c.run()
    assert torch.isneginf(out).all()
    _, _, status = ds.verify_greedy(out, torch.zeros(1, 1, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert status.tolist() == [ds.ST_ZERO_MASS]


@pytest.mark.parametrize("name,value", [("repetition", 0.0), ("repetition", -1.0),
                                        ("repetition", math.nan), ("repetition", math.inf),
                                        ("frequency", math.inf), ("presence", math.nan)])
@pytest.mark.parametrize("inplace", [False, True])
def test_bad_penalties_refuse_their_request(name, value, inplace):
    c = Case(3, 2, 4500, masks=2)
    c.kw[name][1] = value
    x = c.x.cuda()
    out, status = c.run(x, out=x if inplace else None)
    assert status.tolist() == [0, ds.ST_BAD_PENALTY, 0]
    c.check(out)


def test_same_bits_every_time_and_on_another_stream():
    c = Case(4, 6, 9001, torch.bfloat16, history=3000, biases=200, masks=3, tree=True)
    x = c.x.cuda()
    a, _ = c.run(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (None, s, s):
        b, _ = c.run(x, stream=stream)
        assert torch.equal(a, b)


def test_binding_refuses():
    x = torch.zeros(2, 3, 50, device="cuda")
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    for kw in (dict(history=i(2, 5).long(), history_len=i(2)), dict(repetition=i(2)),
               dict(row_mask=i(2, 3))):
        with pytest.raises(TypeError):
            ds.logits_process(x, **kw)
    for kw in (dict(history=i(3, 5), history_len=i(2)), dict(draft_tokens=i(1, 2)),
               dict(mask_words=i(4, 1)), dict(out=torch.zeros(2, 3, 51, device="cuda")),
               dict(mask_words=i(4, 2), mask_rows=i(6))):
        with pytest.raises(ValueError):
            ds.logits_process(x, **kw)
    with pytest.raises(ValueError):
        ds.logits_process(x[0])
    with pytest.raises(RuntimeError):            # a text without its lengths
        ds.logits_process(x, history=i(2, 5))
    with pytest.raises(TypeError):
        ds.logits_process(x.half())
