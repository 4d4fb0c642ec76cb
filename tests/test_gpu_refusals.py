"""What the operators around the prefill turn away, on CUDA tensors: each bad
argument is named, and nothing runs."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    import kimi_delta_attention_kda_gb300 as m
    from kimi_delta_attention_kda_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    m.device_status()
    return m


def bf(*s):
    return torch.zeros(s, dtype=torch.bfloat16, device="cuda")


def f32(*s):
    return torch.zeros(s, device="cuda")


def i32(*s):
    return torch.zeros(s, dtype=torch.int32, device="cuda")


GOOD = {
    "la_prefill": lambda: dict(q=bf(1, 9, 2, 128), k=bf(1, 9, 2, 128), v=bf(1, 9, 4, 128), g=f32(1, 9, 4),
                               init_state=f32(1, 4, 128, 128), out=bf(1, 9, 4, 128),
                               final_state=f32(1, 4, 128, 128)),
    "la_decode": lambda: dict(q=bf(3, 2, 128), k=bf(3, 2, 128), v=bf(3, 4, 128), g=f32(3, 4),
                              state=f32(5, 4, 128, 128), slots=torch.arange(3, dtype=torch.int32, device="cuda"),
                              out=bf(3, 4, 128)),
    "kda_decode": lambda: dict(q=bf(3, 4, 128), k=bf(3, 4, 128), v=bf(3, 4, 128), g=f32(3, 4, 128), beta=bf(3, 4),
                               state=f32(5, 4, 128, 128),
                               slots=torch.arange(3, dtype=torch.int32, device="cuda"), out=bf(3, 4, 128)),
    "gated_norm": lambda: dict(x=bf(7, 128), weight=bf(128), gate=bf(7, 128), out=bf(7, 128)),
    "residual_norm": lambda: dict(x=bf(7, 96), residual=f32(7, 96), weight=bf(96), post_weight=bf(96), gate=bf(96),
                                  out=bf(7, 96), residual_out=f32(7, 96)),
}
OPTIONAL = {"init_state", "out", "final_state", "slots", "gate", "post_weight", "residual_out"}


@pytest.mark.parametrize("op,name", [(op, name) for op, names in {
    "la_prefill": "q k v g init_state out final_state", "la_decode": "q k v g state slots out",
    "kda_decode": "q k v g beta state slots out", "gated_norm": "x weight gate out",
    "residual_norm": "x residual weight post_weight gate out residual_out"}.items() for name in names.split()])
def test_each_argument(kda, op, name):
    call = getattr(kda, op)
    call(**GOOD[op]())
    good = GOOD[op]()[name]
    strided = torch.zeros(good.shape[:-1] + (2 * good.shape[-1],), dtype=good.dtype, device="cuda")[..., ::2]
    bad = [good.double(), good.cpu(), strided, good.new_zeros(good.shape + (1,)),
           good.new_zeros((good.shape[0] + 1,) + good.shape[1:]), good[..., :-1].contiguous()]
    if name in ("x", "state"):
        del bad[4]        # another number of rows is another call
    if op == "residual_norm" and name == "x":
        del bad[-1]
    before = {key: t.clone() for key, t in GOOD[op]().items()}
    for t in bad:
        args = GOOD[op]()
        args[name] = t
        with pytest.raises(ValueError):
            call(**args)
        for key, value in args.items():
            if key != name:
                assert torch.equal(value, before[key])
    if name in OPTIONAL:
        args = GOOD[op]()
        args[name] = None
        call(**args)
    else:
        args = GOOD[op]()
        args[name] = None
        with pytest.raises((ValueError, AttributeError)):
            call(**args)
    torch.cuda.synchronize()
    assert kda.device_status() == 0


def test_values(kda):
    a = GOOD["gated_norm"]()
    with pytest.raises(ValueError, match="activation"):
        kda.gated_norm(**a, activation="relu")
    with pytest.raises(kda.KdaError):
        kda.gated_norm(**a, eps=-1.0)
    with pytest.raises(TypeError):
        kda.gated_norm(**a, eps="small")
    b = GOOD["la_prefill"]()
    del b["init_state"], b["final_state"]
    with pytest.raises(ValueError, match="states"):
        kda.la_prefill(**b, state_dtype=torch.float16)
    with pytest.raises(ValueError, match="cu_seqlens"):
        kda.la_prefill(**b, cu_seqlens=i32(2))
    c = GOOD["la_decode"]()
    c["slots"] = None
    c["state"] = f32(2, 4, 128, 128)
    with pytest.raises(ValueError, match="fewer rows"):
        kda.la_decode(**c)
    d = GOOD["residual_norm"]()
    d["out"] = d["residual_out"]
    with pytest.raises(ValueError, match="out"):
        kda.residual_norm(**d)
    # Overlapping outputs are the library's to refuse.
    e = GOOD["kda_decode"]()
    e["out"] = e["q"]
    with pytest.raises(kda.KdaError):
        kda.kda_decode(**e)
