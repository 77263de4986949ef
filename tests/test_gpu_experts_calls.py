"""GPU tests of the ways to call the operators around experts: through the compiled checks and the
Python ones, with tensors and with raw pointers; every way gives the same bits."""

import pytest

import software_pipelined_tiled_gemm_amd as spg
from tests.test_gpu_feed_forward import _gen, _normal, _t, _workspace

pytestmark = pytest.mark.gpu

T, D, N, E, K = 77, 136, 200, 6, 3


def _pass(as_pointers):
    torch = _t()
    R = T * K
    gen = _gen(3)
    bf = torch.bfloat16
    rand = lambda *s, std=1.0: _normal(gen, s, std).to(bf)
    x, nw, nb, logits = rand(T, D), rand(D), rand(D), _normal(gen, (T, E), 1.0)
    wg, wu, wd, dout = rand(E, N, D, std=0.1), rand(E, N, D, std=0.1), rand(E, D, N, std=0.1), rand(T, D)
    new = lambda *s, dtype=bf: torch.full(s, 7, dtype=dtype, device="cuda")
    out = {"xn": new(T, D), "mean": new(T, dtype=torch.float32), "rstd": new(T, dtype=torch.float32),
           "gate": new(T, K, dtype=torch.float32), "expert": new(T, K, dtype=torch.int32), "slot": new(T, K, dtype=torch.int32),
           "source": new(R, dtype=torch.int32), "offsets": new(E + 1, dtype=torch.int32),
           "h": new(R, N), "g": new(R, N), "u": new(R, N), "y": new(R, D), "out": new(T, D),
           "dy": new(R, D), "dgate": new(T, K, dtype=torch.float32), "dh": new(R, N), "dwd": new(E, D, N),
           "dxr": new(R, D), "dwg": new(E, N, D), "dwu": new(E, N, D), "dxn": new(T, D), "dl": new(T, E, dtype=torch.float32),
           "dx": new(T, D), "dnw": new(D), "dnb": new(D)}
    o = dict(out)
    inputs = [x, nw, nb, logits, wg, wu, wd, dout]
    keep = []
    if as_pointers:
        o = {n: t.data_ptr() for n, t in o.items()}
        x, nw, nb, logits, wg, wu, wd, dout = (t.data_ptr() for t in inputs)

    def ws(plan, **kw):
        w = _workspace(plan.workspace_bytes(**kw))
        keep.append(w)
        return w if w is None or not as_pointers else w.data_ptr()

    torch.cuda.synchronize()                             # raw pointers run on the stream that is given: the default one
    with spg.LayerNorm(T, D) as norm, spg.Router(T, E, K) as route, spg.GroupedGated(R, N, D, E, tokens=T) as up, \
            spg.GroupedGemm(R, D, N, E) as down, spg.Combine(T, K, R, D) as join:
        norm(x, nw, nb, o["xn"], o["mean"], o["rstd"])
        route(logits, o["gate"], o["expert"], o["slot"], o["source"], o["offsets"], workspace=ws(route))
        up(o["xn"], wg, wu, o["offsets"], o["h"], source=o["source"], G=o["g"], U=o["u"], workspace=ws(up))
        down(o["h"], wd, o["offsets"], o["y"], workspace=ws(down))
        join(o["y"], o["slot"], o["gate"], o["out"])
        join.backward(dout, o["y"], o["slot"], o["gate"], o["dy"], o["dgate"])
        down.backward(o["dy"], o["h"], wd, o["offsets"], o["dh"], o["dwd"], workspace=ws(down))
        up.backward(o["dh"], o["xn"], wg, wu, o["g"], o["u"], o["offsets"], o["dxr"], o["dwg"], o["dwu"], source=o["source"],
                    workspace=ws(up))
        join(o["dxr"], o["slot"], None, o["dxn"])
        route.backward(logits, o["expert"], o["dgate"], o["dl"])
        norm.backward(o["dxn"], x, nw, o["mean"], o["rstd"], o["dx"], o["dnw"], o["dnb"], workspace=ws(norm))
        torch.cuda.synchronize()
    assert int(out["offsets"][-1]) == R
    return out


def test_every_way_to_call(monkeypatch):
    torch = _t()
    want = _pass(False)
    ways = {"pointers": _pass(True)}
    with monkeypatch.context() as m:
        m.setattr(spg, "_calls_module", lambda: None)
        ways["Python checks"] = _pass(False)
        ways["Python checks, pointers"] = _pass(True)
    for way, got in ways.items():
        for n, t in want.items():
            assert torch.equal(t, got[n]), (way, n)
    assert all(bool(torch.isfinite(t.float()).all()) for t in want.values())
