"""Host-only checks of the serving operators' C-ABI and Python boundary (no
GPU needed): workspace queries, empty calls, and arguments that are refused
before anything is launched."""
import pytest
import torch

import mixture_experts_routed_sigmoid_b200 as moe
from mixture_experts_routed_sigmoid_b200 import build as moe_build

OK, INVALID, UNSUPPORTED, WS_SMALL = 0, 1, 2, 3
FAKE = 0x10000  # non-null, 256-byte aligned; never dereferenced on rejection


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return moe.load_library()


def _layer(lib, m=4, hidden=64, inter=32, inter_sh=0, top_k=2, E=8, ws=FAKE, ws_bytes=1 << 40, **ptr):
    p = dict(x=FAKE, W_router=FAKE, bias=None, W_gate=FAKE, W_up=FAKE, W_down=FAKE,
             **{k: FAKE if inter_sh else None for k in ("w_sh", "W_sh_gate", "W_sh_up", "W_sh_down")},
             y=FAKE, ids=FAKE, weights=FAKE, logits=FAKE)
    p.update(ptr)
    return lib.moe_layer_decode(*p.values(), m, hidden, inter, inter_sh, top_k, E, ws, ws_bytes, None)


def test_layer_decode_validation(lib):
    assert _layer(lib, m=0) == OK
    assert _layer(lib, m=-1) == INVALID
    assert _layer(lib, m=33) == UNSUPPORTED
    assert b"moe_router_topk" in lib.moe_last_error()      # says what larger batches take
    assert _layer(lib, m=32, top_k=9, E=16) == UNSUPPORTED  # 288 routed rows
    assert _layer(lib, hidden=60) == UNSUPPORTED
    assert _layer(lib, inter=12) == UNSUPPORTED
    assert _layer(lib, inter=0) == UNSUPPORTED
    assert _layer(lib, inter_sh=12) == UNSUPPORTED
    assert _layer(lib, inter_sh=-8) == UNSUPPORTED
    assert _layer(lib, top_k=9) == UNSUPPORTED
    assert _layer(lib, E=1025) == UNSUPPORTED
    for name in ("x", "W_router", "W_gate", "W_up", "W_down", "y", "ids", "weights", "logits"):
        assert _layer(lib, **{name: None}) == INVALID
        assert name.encode() in lib.moe_last_error()
    for name in ("x", "W_router", "W_gate", "W_up", "W_down", "y"):
        assert _layer(lib, **{name: FAKE + 8}) == INVALID
    for name in ("w_sh", "W_sh_gate", "W_sh_up", "W_sh_down"):
        assert _layer(lib, inter_sh=16, **{name: None}) == INVALID
        assert _layer(lib, **{name: FAKE}) == INVALID       # given, but no shared expert
    assert _layer(lib, ws=FAKE + 16) == INVALID
    need = lib.moe_layer_decode_workspace(4, 64, 32, 0, 2, 8)
    assert _layer(lib, ws_bytes=need - 1) == WS_SMALL


def test_layer_decode_workspace(lib):
    f = lib.moe_layer_decode_workspace
    # the activation as three bf16 parts, the scores, the down outputs of every slot
    fixed = 3 * 2 * (16 * 8 * 768 + 16 * 512) + 4 * 16 * 128 + 4 * 16 * 9 * 2048
    assert fixed <= f(16, 2048, 768, 512, 8, 128) < fixed + 4096
    assert f(33, 64, 32, 0, 1, 8) == 0 and f(4, 60, 32, 0, 2, 8) == 0 and f(4, 64, 32, 4, 2, 8) == 0
    assert f(0, 64, 32, 0, 2, 8) > 0


def _lora(lib, m=100, n=32, k=64, rank=16, D=4, dtype=0, ws=FAKE, ws_bytes=1 << 40, **ptr):
    p = dict(x=FAKE, W=FAKE, adapter_ids=FAKE, A=FAKE, B=FAKE, scales=None, y=FAKE)
    p.update(ptr)
    return lib.moe_matmul_lora(*p.values(), dtype, m, n, k, rank, D, ws, ws_bytes, None)


@pytest.mark.parametrize("m", [4, 100])
def test_matmul_lora_validation(lib, m):
    assert _lora(lib, m=0) == OK
    assert _lora(lib, m=-1) == INVALID
    assert _lora(lib, m=(1 << 24) + 1) == UNSUPPORTED
    assert _lora(lib, m=m, n=0) == UNSUPPORTED
    assert _lora(lib, m=m, k=60) == UNSUPPORTED
    assert _lora(lib, m=m, rank=0) == UNSUPPORTED
    assert _lora(lib, m=m, rank=12) == UNSUPPORTED
    assert _lora(lib, m=m, rank=136) == UNSUPPORTED
    assert _lora(lib, m=m, D=0) == UNSUPPORTED
    assert _lora(lib, m=m, D=65537) == UNSUPPORTED
    assert _lora(lib, m=m, dtype=2) == INVALID
    for name in ("x", "W", "adapter_ids", "A", "B", "y"):
        assert _lora(lib, m=m, **{name: None}) == INVALID
        assert name.encode() in lib.moe_last_error()
        assert _lora(lib, m=m, **{name: FAKE + 2}) == INVALID
    assert _lora(lib, m=m, scales=FAKE + 2) == INVALID
    assert _lora(lib, m=m, ws=FAKE + 16) == INVALID
    need = lib.moe_matmul_lora_workspace(m, 32, 64, 16, 4)
    assert need > 0 and _lora(lib, m=m, ws_bytes=need - 1) == WS_SMALL
    assert lib.moe_matmul_lora_workspace(0, 32, 64, 16, 4) > 0


@pytest.mark.parametrize("dtype, elem", [(0, 4), (1, 2)])
def test_matmul_lora_refuses_an_output_over_its_input(lib, dtype, elem):
    x, rows, k, n = 1 << 20, 100, 64, 32
    for y in (x, x + 16, x + rows * k * 2 - 16, x - rows * n * elem + 16):
        assert _lora(lib, x=x, y=y, k=k, n=n, dtype=dtype) == INVALID
        assert b"overlaps" in lib.moe_last_error()
    for y in (x + rows * k * 2, x - rows * n * elem):  # side by side: only the workspace is refused
        assert _lora(lib, x=x, y=y, k=k, n=n, dtype=dtype, ws_bytes=0) == WS_SMALL


def test_python_boundary_refuses_before_the_library():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_layer_decode(bf(2, 64), bf(4, 64), None, 2, bf(4, 32, 64), bf(4, 32, 64), bf(4, 64, 32))
    with pytest.raises(TypeError):
        moe.moe_layer_decode(torch.zeros(2, 64), bf(4, 64), None, 2, bf(4, 32, 64), bf(4, 32, 64), bf(4, 64, 32))
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_matmul_lora(bf(2, 64), bf(8, 64), torch.zeros(2, dtype=torch.int32), bf(1, 8, 64), bf(1, 8, 8))
    with pytest.raises(TypeError):
        moe.moe_matmul_lora(torch.zeros(2, 64), bf(8, 64), torch.zeros(2, dtype=torch.int32), bf(1, 8, 64), bf(1, 8, 8))
