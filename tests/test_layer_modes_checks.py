"""What PoetxLinear and Int8Linear do on the host around the C calls: refusals
that leave a layer as it was, where their scratch comes from and on which
stream and device the calls run.  The C calls are stood in for, so no GPU is
needed."""
import pytest
import torch

import orthogonal_equivalence_b200 as px
from orthogonal_equivalence_b200 import layer as layer_py

BF = torch.bfloat16


@pytest.mark.parametrize("scratch,match", [(torch.empty(128 * 192 - 1, dtype=BF), "elements"),
                                           (torch.empty(128 * 192), "scratch: dtype"),
                                           (torch.empty(128, 192, dtype=BF), "scratch: shape")])
def test_a_refused_scratch_leaves_the_layer_as_it_was(monkeypatch, scratch, match):
    monkeypatch.setattr(layer_py, "poetx_weight_quantize", lambda *a: None)
    L = px.PoetxLinear(128, 192, 64, px.POETX_BF16, device="cpu")
    W = L.W
    with pytest.raises(ValueError, match=match):
        L.quantize_weight(scratch)
    assert L.W is W and L.Wq is None and L.Wscale is None


class Streams:
    """torch's streams stood in for: allocations note the stream that is current."""

    def __init__(self, monkeypatch, capturing):
        self.current, self.made = "current", []
        empty = torch.empty

        class On:
            def __init__(on, s):
                on.s = s

            def __enter__(on):
                on.was = self.current
                self.current = on.s or on.was

            def __exit__(on, *a):
                self.current = on.was

        def made(*a, device=None, **k):
            t = empty(*a, **k)
            self.made.append((t, self.current))
            return t

        monkeypatch.setattr(torch.cuda, "stream", On)
        monkeypatch.setattr(torch.cuda, "device", lambda d: On(None))
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)
        monkeypatch.setattr(torch, "empty", made)
        monkeypatch.setattr(layer_py, "_torch_stream", lambda s, device: s, raising=False)


@pytest.mark.parametrize("capturing", [False, True])
def test_scratch_belongs_to_the_stream_that_uses_it(monkeypatch, capturing):
    # freed scratch (a captured call's at its end, an eager one's when a larger one takes its place) goes back to
    # the stream it was made on: another one than the call's could hand it out while the call still runs
    s = Streams(monkeypatch, capturing)
    cuda, held = torch.device("cuda", 0), {}
    layer_py._workspace(held, "fwd", 100, cuda, "side")
    layer_py._workspace(held, "fwd", 200, cuda, "side")
    layer_py._workspace(held, "bwd", 100, cuda, None)
    assert [(t.numel(), on) for t, on in s.made] == [(100, "side"), (200, "side"), (100, "current")]
    assert not capturing or not held


def test_every_call_asks_for_scratch_on_its_stream(monkeypatch):
    L = px.PoetxLinear(128, 192, 64, px.POETX_BF16, device="cpu")
    group = px.LayerGroup([L])
    group.flatten_params()
    asked = []
    workspace = layer_py._workspace
    monkeypatch.setattr(layer_py, "_workspace", lambda *a: (asked.append(a[1:2] + a[4:]), workspace(*a[:4]))[1])
    for name in ("poetx_forward", "poetx_backward", "poetx_backward_dG", "poetx_layer_cnp_build", "poetx_merge",
                 "poetx_layers_cnp_build", "poetx_cnp_backward", "poetx_frame_import"):
        monkeypatch.setattr(layer_py, name, lambda *a: None)
    x, dz = torch.zeros(4, 128, dtype=BF), torch.zeros(4, 192, dtype=BF)
    dG = group.dG_buffer()
    L.forward(x, stream="side")
    L.backward(x, None, dz, stream="side")
    L.backward_dG(x, None, dz, *group.dG_views(dG)[0], stream="side")
    L.build(stream="side")
    L.merge(L.permR, L.permP, stream="side")
    group.build(stream="side")
    group.cnp_backward(dG, torch.zeros_like(group.q), stream="side")
    assert asked == [(k, "side") for k in ("fwd", "bwd", "bwd", "cnp", "merge", "build", "bwd")]


def test_the_context_of_a_call_switches_to_its_device_and_stream(monkeypatch):
    s, seen = object(), []
    monkeypatch.setattr(layer_py, "_torch_stream", lambda stream, device: stream)
    monkeypatch.setattr(torch.cuda, "device", lambda d: seen.append(("device", d)))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: seen.append(("stream", s)))   # (switches the device as well)
    for stream in (None, s):
        layer_py._on(stream, torch.device("cuda", 1))
    layer_py._on(None, torch.device("cpu"))
    assert seen == [("device", torch.device("cuda", 1)), ("stream", s)]


@pytest.mark.parametrize("form", ["full", "codes", "int8_product"])
def test_every_call_of_a_layer_runs_on_its_device(monkeypatch, form):
    # a layer on another device than the current one: each C call, the expansion of a quantized weight among
    # them, is made inside the context of the layer's device
    inside, calls = [], []

    class On:
        def __init__(on, stream, device):
            on.at = (stream, device.type)

        def __enter__(on):
            inside.append(on.at)

        def __exit__(on, *a):
            inside.pop()

    monkeypatch.setattr(layer_py, "_on", On)
    names = [n for n in dir(layer_py) if n.startswith("poetx_") and not n.endswith("_bytes")]
    for name in names:
        monkeypatch.setattr(layer_py, name, lambda *a, name=name: calls.append((name, inside[-1] if inside else None)))
    L = px.PoetxLinear(128, 192, 64, px.POETX_BF16, device="cpu")
    group = px.LayerGroup([L])
    q = group.flatten_params()
    dG = group.dG_buffer()
    x, dz = torch.zeros(4, 128, dtype=BF), torch.zeros(4, 192, dtype=BF)
    if form != "full":
        L.quantize_weight(stream="s", int8_product=form == "int8_product")
    for save8 in (False, True):
        _, saved = L.forward(x, save8=save8, stream="s")
        L.backward(x, saved, dz, stream="s")
        L.backward_dG(x, saved, dz, *group.dG_views(dG)[0], stream="s")
    if form != "int8_product":
        L.export_weight(stream="s")
        L.merge(L.permR, L.permP, stream="s")
    group.cnp_backward(dG, torch.zeros_like(q), stream="s")
    group.optimizer_step(torch.zeros_like(q), 1e-3, stream="s")
    L.load(L.W.new_zeros(192, 128, dtype=BF), L.permR, L.permP, L.qR, L.qP, stream="s")
    assert {at for _, at in calls} == {("s", "cpu")}
    want = {"poetx_forward_q8", "poetx_backward_q8", "poetx_backward_dG_q8", "poetx_cnp_backward", "poetx_adamw_step",
            "poetx_layers_cnp_build", "poetx_frame_import", "poetx_layer_cnp_build"}
    want |= {"full": {"poetx_merge"}, "codes": {"poetx_merge", "poetx_weight_dequantize"}, "int8_product": set()}[form]
    assert want <= {name for name, _ in calls}
