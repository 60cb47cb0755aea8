"""Rotation, latent write and latent attention refuse a tensor of another
device than the current one, whichever argument it is.  The tensors here are
the host's and only say that they lie on a CUDA device; the library's entry
is replaced by one that notes the call -- no GPU needed."""
import pytest
import torch

import draft_sampling_verification_gb300 as ds

F32, BF16, I32, I64 = torch.float32, torch.bfloat16, torch.int32, torch.int64


class Current(torch.Tensor):
    is_cuda = True

    def get_device(self):
        return 0


class Another(Current):
    def get_device(self):
        return 1


def on(kind, *shape, dtype=BF16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(kind)


def tensors(**shapes):
    """name -> (shape, dtype); bf16 where none is given."""
    return {k: v if isinstance(v, tuple) and isinstance(v[1], torch.dtype) else (v, BF16)
            for k, v in shapes.items()}


HEADS = tensors(q=(4, 2, 64), k=(4, 1, 64), positions=((4,), I32), table=((32,), I64),
                q_weight=((64,), F32), k_weight=((64,), F32))
PAGED = tensors(v=(4, 1, 64), k_cache=(2, 8, 1, 64), v_cache=(2, 8, 1, 64), slots=((4,), I32))
LATENT = tensors(c=(4, 128), k_rope=(4, 64), positions=((4,), I32), table=((32,), I64),
                 cache=(2, 8, 192), slots=((4,), I32), rows=((4,), I32), weight=((128,), F32))
SEEN = tensors(q=(1, 2, 4, 192), cache=(2, 8, 192), block_table=((1, 2), I32), ctx_len=((1,), I32),
               n_nodes=((1,), I32), tree_mask=((1, 2), I64))
TURN = dict(eps=1e-6, rot_start=0, interleaved=False, magnitude=1.0)
BYTES = 16 << 20  # of the workspace

CALLS = {
    "qk_rotate": (ds.qk_rotate, HEADS, {}),
    "dspark_qk_rotate": (ds.dspark_qk_rotate,
                         {**HEADS, **tensors(q_out=(4, 2, 64), k_out=(4, 1, 64))}, TURN),
    "rotate_write": (ds.rotate_write, {**HEADS, **PAGED}, {}),
    "rotate_write by rows": (ds.rotate_write, {
        **{k: v for k, v in HEADS.items() if k not in ("q", "q_weight")}, **PAGED,
        **tensors(rows=((4,), I32))}, dict(q=None)),
    "dspark_rotate_write": (ds.dspark_rotate_write, {
        **HEADS, **PAGED, **tensors(q_out=(4, 2, 64))}, dict(rows=None, **TURN)),
    "latent_write": (ds.latent_write, LATENT, {}),
    "dspark_latent_write": (ds.dspark_latent_write, LATENT, dict(
        eps=1e-6, interleaved=False, magnitude=1.0)),
    "latent_attention": (ds.latent_attention, SEEN, dict(latent_dim=128, scale=0.1)),
    "dspark_latent_attention": (ds.dspark_latent_attention, {
        **SEEN, **tensors(out=(1, 2, 4, 128), lse=((1, 2, 4), F32), req_status=((1,), I32),
                          workspace=((BYTES,), torch.uint8))}, dict(latent_dim=128, scale=0.1)),
}


@pytest.fixture
def called(monkeypatch):
    calls = []
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(ds, "_stream", lambda stream: None)
    monkeypatch.setattr(ds, "_call", lambda name, *args: calls.append(name))
    monkeypatch.setattr(ds, "dspark_latent_attention_workspace_bytes", lambda *args: BYTES)
    return calls


@pytest.mark.parametrize("name,argument", [(n, a) for n, (_, t, _) in CALLS.items()
                                           for a in [None, *t]])
def test_each_argument(called, name, argument):
    f, shapes, others = CALLS[name]
    args = {k: on(Another if k == argument else Current, *shape, dtype=dtype)
            for k, (shape, dtype) in shapes.items()}
    if argument is None:
        f(**args, **others)
        assert len(called) == 1
        return
    with pytest.raises(ValueError, match="current CUDA device"):
        f(**args, **others)
    assert called == []


@pytest.mark.parametrize("argument", ["q_out", "k_out"])
def test_given_outputs(called, argument):
    args = {k: on(Current, *shape, dtype=dtype) for k, (shape, dtype) in HEADS.items()}
    out = {k: on(Another if k == argument else Current, *s)
           for k, s in (("q_out", (4, 2, 64)), ("k_out", (4, 1, 64)))}
    with pytest.raises(ValueError, match="current CUDA device"):
        ds.qk_rotate(**args, out=(out["q_out"], out["k_out"]))
    if argument == "q_out":
        args.update({k: on(Current, *shape, dtype=dtype) for k, (shape, dtype) in PAGED.items()})
        with pytest.raises(ValueError, match="current CUDA device"):
            ds.rotate_write(**args, out=out["q_out"])
    assert called == []


def test_what_is_not_looked_at(called):
    """Without keys or queries, what belongs to them may lie anywhere."""
    args = {k: on(Current, *shape, dtype=dtype) for k, (shape, dtype) in HEADS.items()}
    weight, out = on(Another, 64, dtype=F32), on(Another, 4, 1, 64)
    ds.qk_rotate(**{**args, "k": None, "k_weight": weight}, out=(args["q"], out))
    ds.qk_rotate(**{**args, "q": None, "q_weight": weight}, out=(out, args["k"]))
    paged = {k: on(Current, *shape, dtype=dtype) for k, (shape, dtype) in PAGED.items()}
    ds.rotate_write(**{**args, **paged, "q": None, "q_weight": weight})
    assert called == ["dspark_qk_rotate"] * 2 + ["dspark_rotate_write"]
