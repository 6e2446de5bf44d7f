"""libmoe_block.so on the host: its header's symbols, and every refusal of the C ABI and of the
Python binding. Nothing here reaches the HIP runtime: each call fails its checks or has
nothing to do, and the addresses are never dereferenced."""
import ctypes
import glob
import os
import re
import subprocess

import pytest
import torch

import memory_bound_elementwise_amd as mbe
from memory_bound_elementwise_amd import build as mbuild
from memory_bound_elementwise_amd.moe_block import load_library

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, ALIGN = 0, 1, 2
BF16, F16, F32 = 0, 1, 2
A = 1 << 20            # an aligned address; tensors lie 2^40 apart
NAN, INF = float("nan"), float("inf")


def at(i):
    return A + (i << 40)


def test_header_symbols_are_exported():
    heads = sorted(os.path.basename(h) for h in glob.glob(os.path.join(ROOT, "include", "block", "*.h")))
    assert heads == ["moe_block.h"]
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "block", "moe_block.h")).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:const\s+)?[a-z_0-9]+\s*\*?\s*\b([a-z_0-9]+)\s*\(", text, flags=re.M))
    load_library()
    nm = subprocess.run(["nm", "-D", "--defined-only", mbuild.lib_path("moe_block")], capture_output=True, text=True).stdout
    exported = set(re.findall(r" T ((?:block|moe_block)_\w+)$", nm, flags=re.M))
    assert names and names == exported
    from memory_bound_elementwise_amd.moe_block import _SIGS
    assert set(_SIGS) == names


def test_header_is_plain_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "block/moe_block.h"\nint main(void) { return (int)BLOCK_OK; }\n')
    res = subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-D__HIP_PLATFORM_AMD__", f"-I{ROOT}/include",
                          "-isystem", os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "include"), "-fsyntax-only",
                          str(src)], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr


def test_status_strings_and_version():
    lib = load_library()
    assert lib.moe_block_abi_version() == 1
    texts = [lib.moe_block_status_string(i) for i in range(5)]
    assert len(set(texts)) == 5 and all(texts)


def norm_fwd(x=at(0), w=at(1), b=at(2), y=at(3), mean=at(4), rstd=at(5), rows=4, cols=24, eps=1e-5, dt=BF16, wt=F32):
    return load_library().block_layer_norm_fwd(x, w, b, y, mean, rstd, rows, cols, eps, dt, wt, None)


def test_layer_norm_fwd_refusals():
    assert norm_fwd(rows=0) == OK and norm_fwd(rows=0, x=None, y=None) == OK
    for bad in (dict(rows=-1), dict(cols=0), dict(cols=-8), dict(cols=(1 << 20) + 1), dict(rows=1 << 46), dict(eps=-1.0),
                dict(eps=NAN), dict(eps=INF), dict(dt=3), dict(dt=-1), dict(wt=F16), dict(dt=F32, wt=BF16), dict(x=None),
                dict(y=None), dict(mean=None), dict(rstd=None), dict(y=at(0)), dict(y=at(0) + 16), dict(y=at(1)),
                dict(y=at(2) - 32), dict(mean=at(0) + 4), dict(rstd=at(4)), dict(mean=at(3))):
        assert norm_fwd(**bad) == INVALID, bad
    for bad in (dict(x=A + 2), dict(y=at(3) + 8), dict(w=at(1) + 4), dict(b=at(2) + 2), dict(mean=at(4) + 2),
                dict(rstd=at(5) + 1)):
        assert norm_fwd(**bad) == ALIGN, bad


def norm_bwd(gy=at(0), x=at(1), w=at(2), mean=at(3), rstd=at(4), gx=at(5), gw=at(6), gb=at(7), rows=4, cols=24, dt=BF16,
             wt=F32, ws=at(8), size=1 << 30):
    return load_library().block_layer_norm_bwd(gy, x, w, mean, rstd, gx, gw, gb, rows, cols, dt, wt, ws, size, None)


def test_layer_norm_bwd_refusals():
    assert norm_bwd(rows=0, gw=None, gb=None) == OK
    assert norm_bwd(rows=0, gw=None, gb=None, x=None, gy=None, mean=None, rstd=None, ws=None, size=0) == OK
    need = load_library().block_layer_norm_bwd_workspace(4, 24)
    assert need > 0
    for bad in (dict(rows=-1), dict(cols=0), dict(dt=7), dict(wt=F16), dict(gy=None), dict(x=None), dict(mean=None),
                dict(rstd=None), dict(ws=None), dict(size=need - 1), dict(size=0), dict(gx=at(0)), dict(gx=at(1)),
                dict(gw=at(2)), dict(gw=at(7)), dict(ws=at(1)), dict(ws=at(5)), dict(gb=at(3))):
        assert norm_bwd(**bad) == INVALID, bad
    for bad in (dict(gy=A + 2), dict(x=at(1) + 4), dict(gx=at(5) + 8), dict(gw=at(6) + 4), dict(ws=at(8) + 4),
                dict(mean=at(3) + 2)):
        assert norm_bwd(**bad) == ALIGN, bad
    for rows, cols in ((-1, 8), (8, 0), (8, 1 << 21), (1 << 47, 8)):
        assert load_library().block_layer_norm_bwd_workspace(rows, cols) == 0


def linear(x=at(0), w=at(1), b=at(2), r=at(3), y=at(4), m=4, n=16, k=24, act=1, dt=BF16, ws=at(5), size=1 << 36):
    return load_library().block_linear_act(x, w, b, r, y, m, n, k, act, dt, ws, size, None)


def test_linear_refusals():
    assert linear(m=0) == OK and linear(m=0, x=None, w=None, y=None) == OK
    for bad in (dict(m=-1), dict(n=0), dict(k=0), dict(n=-8), dict(m=(1 << 24) + 1), dict(n=(1 << 20) + 8),
                dict(k=(1 << 20) + 8), dict(m=1 << 20, n=1 << 17), dict(m=1 << 20, k=1 << 17),
                dict(n=1 << 19, k=1 << 19), dict(act=4), dict(act=-1), dict(act=9), dict(dt=F32), dict(dt=5), dict(x=None),
                dict(w=None), dict(y=None), dict(y=at(0)), dict(y=at(1) + 16), dict(y=at(2)), dict(y=at(3))):
        assert linear(**bad) == INVALID, bad
    for bad in (dict(n=12), dict(k=20), dict(x=A + 2), dict(w=at(1) + 8), dict(b=at(2) + 2), dict(r=at(3) + 4),
                dict(y=at(4) + 2)):
        assert linear(**bad) == ALIGN, bad


def test_linear_short_workspace():
    """Wherever a workspace is needed, one byte less is refused."""
    lib = load_library()
    for m, n, k in ((100, 64, 7168), (8, 64, 1 << 16), (4096, 4096, 4096)):
        need = lib.block_linear_act_workspace(m, n, k)
        if need:
            assert linear(m=m, n=n, k=k, size=need - 1) == INVALID
            assert linear(m=m, n=n, k=k, ws=None) == INVALID
            assert linear(m=m, n=n, k=k, ws=at(0)) == INVALID
            assert linear(m=m, n=n, k=k, ws=at(5) + 4) == ALIGN
    assert lib.block_linear_act_workspace(-1, 8, 8) == 0 and lib.block_linear_act_workspace(4, 0, 8) == 0


def route(x=at(0), w=at(1), rdt=BF16, ids=at(2), probs=at(3), tokens=4, hidden=64, experts=8, k=2, valid=None, ws=at(4),
          size=1 << 30):
    return load_library().block_moe_route(x, w, rdt, ids, probs, tokens, hidden, experts, k, 0, valid, ws, size, None)


def test_route_refusals():
    need = load_library().block_moe_route_workspace(4, 64, 8)
    assert need > 0 and route(tokens=0) == OK
    for bad in (dict(tokens=-1), dict(tokens=(1 << 19) + 1), dict(hidden=0), dict(hidden=(1 << 20) + 8), dict(experts=0),
                dict(experts=1025), dict(k=0), dict(k=9), dict(k=65, experts=128), dict(rdt=F16), dict(x=None),
                dict(w=None), dict(ids=None), dict(probs=None), dict(ws=None), dict(size=need - 1), dict(ids=at(0)),
                dict(probs=at(2)), dict(ws=at(1)), dict(valid=at(2))):
        assert route(**bad) == INVALID, bad
    for bad in (dict(hidden=60), dict(x=A + 2), dict(w=at(1) + 8), dict(ids=at(2) + 2), dict(probs=at(3) + 1),
                dict(valid=at(6) + 2), dict(ws=at(4) + 8)):
        assert route(**bad) == ALIGN, bad


def experts(x=at(0), wu=at(1), wd=at(2), ids=at(3), probs=at(4), r=at(5), y=at(6), ydt=BF16, tokens=4, hidden=64,
            inter=24, n=8, k=2, act=4, limit=7.0, valid=None, ws=at(7), size=1 << 30):
    return load_library().block_moe_experts(x, wu, wd, ids, probs, r, y, ydt, tokens, hidden, inter, n, k, act, limit,
                                            valid, ws, size, None)


def layer(x=at(0), rw=at(8), rdt=BF16, wu=at(1), wd=at(2), ids=at(3), probs=at(4), r=at(5), y=at(6), ydt=BF16, tokens=4,
          hidden=64, inter=24, n=8, k=2, act=4, limit=7.0, valid=None, ws=at(7), size=1 << 30):
    return load_library().block_moe_layer(x, rw, rdt, wu, wd, r, y, ydt, ids, probs, tokens, hidden, inter, n, k, 0, act,
                                          limit, valid, ws, size, None)


@pytest.mark.parametrize("call", [experts, layer])
def test_expert_refusals(call):
    lib = load_library()
    need = (lib.block_moe_experts_workspace(4, 64, 24, 8, 2) if call is experts else
            lib.block_moe_layer_workspace(4, 64, 24, 8, 2))
    assert need > 0 and call(tokens=0) == OK
    for bad in (dict(tokens=-1), dict(tokens=513), dict(tokens=1 << 40), dict(hidden=0), dict(inter=0),
                dict(hidden=(1 << 16) + 8), dict(inter=(1 << 16) + 8), dict(n=0), dict(n=1025), dict(k=0), dict(k=1025),
                dict(act=0), dict(act=1), dict(act=5), dict(limit=0.0), dict(limit=-1.0), dict(limit=NAN), dict(ydt=F16),
                dict(ydt=3), dict(x=None), dict(wu=None), dict(wd=None), dict(ids=None), dict(probs=None), dict(y=None),
                dict(ws=None), dict(size=need - 1), dict(y=at(0)), dict(y=at(5)), dict(y=at(2) + 16), dict(y=at(1)),
                dict(y=at(3) - 16), dict(ws=at(6)), dict(ws=at(0)), dict(valid=at(6))):
        assert call(**bad) == INVALID, bad
    for bad in (dict(hidden=60), dict(inter=20), dict(x=A + 2), dict(wu=at(1) + 8), dict(wd=at(2) + 4), dict(r=at(5) + 2),
                dict(y=at(6) + 8), dict(ids=at(3) + 2), dict(probs=at(4) + 2), dict(valid=at(9) + 1), dict(ws=at(7) + 8)):
        assert call(**bad) == ALIGN, bad


def test_layer_refusals_of_its_router():
    for bad in (dict(k=9), dict(rdt=F16), dict(rw=None), dict(ids=at(0)), dict(probs=at(3)), dict(ids=at(8)),
                dict(n=100, k=65)):
        assert layer(**bad) == INVALID, bad
    assert layer(rw=at(8) + 2) == ALIGN


def test_exports():
    for name in ("layer_norm_fwd", "layer_norm_bwd", "LayerNorm", "linear_act", "moe_route", "moe_experts", "moe_layer"):
        assert name in mbe.__all__ and callable(getattr(mbe, name))


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_checks_layer_norm():
    x, w, f = _t(4, 24), _t(24), torch.float32
    st = _t(4, dtype=f)
    with pytest.raises(ValueError, match="GPU"):
        mbe.layer_norm_fwd(x, w, w, _t(4, 24))
    for bad in ((x[0], w, w, x), (x, _t(23), w, x), (x, w, _t(25), x), (x, w, w, _t(4, 23)), (x.t(), w, w, x.t()),
                (x, w, w, x, st), (x, w, w, x, st, _t(5, dtype=f))):
        with pytest.raises(ValueError):
            mbe.layer_norm_fwd(*bad)
    for bad in ((_t(4, 24, dtype=torch.int16), w, w, x), (x, _t(24, dtype=torch.float16), None, x),
                (x, w, _t(24, dtype=f), x), (x, w, w, _t(4, 24, dtype=f)), (x, w, w, x, _t(4), _t(4))):
        with pytest.raises(TypeError):
            mbe.layer_norm_fwd(*bad)
    with pytest.raises(ValueError):
        mbe.layer_norm_bwd(_t(3, 24), x, w, st, st, x, w, w)
    with pytest.raises(TypeError):
        mbe.layer_norm_bwd(x, x, w, st, st, x, _t(24, dtype=f), w)
    with pytest.raises(ValueError, match="GPU"):
        mbe.layer_norm_bwd(x, x, w, st, st, x, w, w)


def test_binding_checks_products():
    x, w, y = _t(4, 24), _t(16, 24), _t(4, 16)
    with pytest.raises(ValueError, match="GPU"):
        mbe.linear_act(x, w, y)
    for bad in (dict(weight=_t(16, 32)), dict(y=_t(4, 24)), dict(bias=_t(15)), dict(residual=_t(4, 24)),
                dict(activation="relu"), dict(x=_t(4, 24, 1))):
        kw = dict(x=x, weight=w, y=y) | bad
        with pytest.raises(ValueError):
            mbe.linear_act(**kw)
    for bad in (dict(weight=_t(16, 24, dtype=torch.float16)), dict(y=_t(4, 16, dtype=torch.float32)),
                dict(x=_t(4, 24, dtype=torch.float32))):
        kw = dict(x=x, weight=w, y=y) | bad
        with pytest.raises(TypeError):
            mbe.linear_act(**kw)
    with pytest.raises(RuntimeError, match="no_grad"):
        mbe.linear_act(x, w.clone().requires_grad_(), y)


def test_binding_checks_experts():
    i32, f32 = torch.int32, torch.float32
    x, rw, wu, wd = _t(4, 24), _t(6, 24), _t(6, 32, 24), _t(6, 24, 16)
    ids, probs = _t(4, 2, dtype=i32), _t(4, 2, dtype=f32)
    good = dict(x=x, w_up=wu, w_down=wd, ids=ids, probs=probs, y=_t(4, 24))
    with pytest.raises(ValueError, match="GPU"):
        mbe.moe_experts(**good)
    for bad in (dict(w_up=_t(6, 16, 24)), dict(w_up=_t(5, 32, 24)), dict(w_down=_t(6, 24)), dict(probs=_t(4, 3, dtype=f32)),
                dict(ids=_t(3, 2, dtype=i32)), dict(y=_t(4, 25)), dict(activation="silu"), dict(limit=0.0),
                dict(limit=NAN), dict(residual=_t(3, 24)), dict(valid_tokens=_t(2, dtype=i32))):
        with pytest.raises(ValueError):
            mbe.moe_experts(**(good | bad))
    for bad in (dict(x=_t(4, 24, dtype=torch.float16)), dict(ids=_t(4, 2, dtype=torch.int64)), dict(probs=_t(4, 2)),
                dict(y=_t(4, 24, dtype=torch.float16)), dict(valid_tokens=_t(1, dtype=torch.int64))):
        with pytest.raises(TypeError):
            mbe.moe_experts(**(good | bad))
    with pytest.raises(ValueError, match="GPU"):
        mbe.moe_layer(x, rw, wu, wd, _t(4, 24), ids, probs)
    with pytest.raises(ValueError):
        mbe.moe_layer(x, _t(5, 24), wu, wd, _t(4, 24), ids, probs)
    with pytest.raises(ValueError, match="GPU"):
        mbe.moe_route(x, rw, ids, probs)
    with pytest.raises(TypeError):
        mbe.moe_route(x, rw.to(torch.float16), ids, probs)
    with pytest.raises(ValueError):
        mbe.moe_route(x, rw, ids, _t(4, 3, dtype=f32))
