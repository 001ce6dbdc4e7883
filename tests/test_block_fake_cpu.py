"""Host logic of the block operators' C entry points over fake devices (CPU)."""
import pytest

import fake_device
from expert_routed_ffn_gemm_gb300 import binding

INVALID, UNSUPPORTED, OK = binding.MOE_ERR_INVALID_ARG, binding.MOE_ERR_UNSUPPORTED, binding.MOE_OK


@pytest.fixture(scope="module")
def lib():
    return fake_device.load()


@pytest.mark.parametrize("rows,n,status", [(1 << 27, 1 << 20, UNSUPPORTED), (1 << 30, 1 << 20, UNSUPPORTED),
                                           (120 << 20, 1 << 20, UNSUPPORTED), (119 << 20, 1 << 20, OK),
                                           (1 << 30, 1 << 16, OK)])
@pytest.mark.parametrize("gated", [0, 1])
def test_products_of_more_than_2_31_tiles_are_refused(lib, rows, n, status, gated):
    """Work items are numbered in 32 bits: 240 token rows by 256 weight rows each at these sizes.  One group of 2^27
    rows has 559,241 x 4096 of them."""
    h = fake_device.experts(lib, 1, n, 32, gated)
    p = fake_device.address(0)
    before = fake_device.value(lib, "fake_launches")
    assert lib.moe_mx4_matmul(h, p, p, rows, p, p, None, p, 0, 1, None) == status
    assert fake_device.value(lib, "fake_launches") == before + (status == OK)
    lib.moe_mx4_free(h)


def calls(lib):
    """name: (function of its buffers, the buffers' names) of every entry that launches."""
    import ctypes

    cfg = ctypes.byref(binding.moe_norm_config(0, 0, 1, 0, 0, 1.0, 1e-6))
    h = fake_device.experts(lib, 2, 64, 64, 0, device=0)
    return h, {
        "quantize": (lambda b: lib.moe_mx4_quantize(b["x"], 0, 4, 64, b["src"], 1, 4, b["codes"], b["scales"], b["values"],
                                                    None), ("x", "src", "codes", "scales", "values")),
        "gather": (lambda b: lib.moe_mx4_gather(b["codes"], b["scales"], 4, 64, b["src"], 1, 4, b["out"], b["out_scales"],
                                                None), ("codes", "scales", "src", "out", "out_scales")),
        "matmul": (lambda b: lib.moe_mx4_matmul(h, b["codes"], b["scales"], 4, b["offsets"], b["out_rows"],
                                                b["row_scale"], b["out"], 0, 4, None),
                   ("codes", "scales", "offsets", "out_rows", "row_scale", "out")),
        "norm": (lambda b: lib.moe_norm_residual(cfg, 2, 64, b["x"], b["y"], 1, b["w_post"], b["gate"], b["w_pre"],
                                                 b["out"], b["n"], None),
                 ("x", "y", "w_post", "gate", "w_pre", "out", "n")),
        "backward": (lambda b: lib.moe_norm_residual_backward(
            cfg, 2, 64, b["d_out"], b["d_n"], b["out"], b["y"], 1, b["w_post"], b["gate"], b["w_pre"], b["dx"], b["dy"],
            b["d_w_post"], b["d_gate"], b["d_w_pre"], b["workspace"], 1 << 30, None),
            ("d_out", "d_n", "out", "y", "w_post", "gate", "w_pre", "dx", "dy", "d_w_post", "d_gate", "d_w_pre",
             "workspace")),
        "backward of no tokens": (lambda b: lib.moe_norm_residual_backward(
            cfg, 0, 64, None, None, None, None, 1, None, None, None, None, None, b["d_w_post"], b["d_gate"], b["d_w_pre"],
            None, 0, None), ("d_w_post", "d_gate", "d_w_pre")),
    }


@pytest.mark.parametrize("name", ["quantize", "gather", "matmul", "norm", "backward", "backward of no tokens"])
def test_buffers_of_two_devices_are_refused(lib, name):
    """A call whose buffers lie on two devices is turned down before any launch; on one device, whichever is current, it
    is launched there; managed memory goes with any."""
    h, table = calls(lib)
    call, names = table[name]
    here = {k: fake_device.address(0, 4096 * i) for i, k in enumerate(names)}
    for current in (0, 1):
        lib.cudaSetDevice(current)
        assert call(here) == OK and fake_device.value(lib, "fake_launch_device") == 0
        launches = fake_device.value(lib, "fake_launches")
        for k in names:
            assert call({**here, k: fake_device.address(1)}) == INVALID, k
        assert fake_device.value(lib, "fake_launches") == launches
        for k in names:
            assert call({**here, k: fake_device.address(1, managed=True)}) == OK, k
            assert fake_device.value(lib, "fake_launch_device") == 0
    there = {k: fake_device.address(1, 4096 * i) for i, k in enumerate(names)}
    assert call(there) == (INVALID if name == "matmul" else OK)  # the handle's device
    lib.cudaSetDevice(0)
    lib.moe_mx4_free(h)


def test_weights_of_another_device_are_refused(lib):
    import ctypes

    h, cfg = ctypes.c_void_p(), binding.moe_mx4_config(2, 64, 64, 0)
    for current in (0, 1):
        lib.cudaSetDevice(current)
        a, b = fake_device.address(current), fake_device.address(1 - current)
        for codes, scales in ((a, b), (b, a), (b, b)):
            assert lib.moe_mx4_init(ctypes.byref(cfg), codes, scales, ctypes.byref(h)) == INVALID
    lib.cudaSetDevice(0)


def tile_of(lib, counts, n, cols, gated):
    h = fake_device.experts(lib, len(counts), n, cols, int(gated))
    p = fake_device.address(0)
    rows = sum(counts)
    assert lib.moe_mx4_matmul(h, p, p, rows, p, None, None, p, 0, rows, None) == OK
    lib.moe_mx4_free(h)
    return fake_device.value(lib, "fake_tile"), fake_device.value(lib, "fake_balanced")


@pytest.mark.parametrize("gated", [False, True])
def test_sizes_of_the_ring_tests_take_their_tiles(lib, gated):
    """On 152 SMs: each tile with three items to a CTA, or a pair, at least; 32-row tiles in parts; pairs with an odd number
    of weight tiles."""
    import test_mx4_rings_gpu as rings

    for tile, counts in rings.WRAPS.items():
        assert tile_of(lib, counts, rings.WRAP_N, rings.K_LONG, gated)[0] == tile
        items = sum(-(-c // tile) for c in counts) * (rings.WRAP_N // 128) // (2 if tile == 240 else 1)
        assert items >= 3 * (76 if tile == 240 else 152)
    counts, n, cols = rings.PARTS
    assert tile_of(lib, counts, n, cols, gated) == (32, 1)
    for counts, n, cols in rings.PARTS_16:
        assert tile_of(lib, counts, n, cols, gated) == (16, 1)
    for counts, n, g in rings.ODD_TILES:
        assert tile_of(lib, counts, n, rings.ODD_K, g)[0] == 240 and (-(-n // 128)) % 2 == 1


@pytest.mark.parametrize("items,steps,balanced", [
    (24, 16, 0), (24, 23, 0), (24, 24, 1), (48, 48, 1), (52, 24, 0), (88, 48, 0), (128, 16, 0), (128, 64, 0), (152, 64, 0),
    (160, 8, 0), (180, 8, 0), (160, 16, 1), (180, 10, 1), (180, 16, 1), (200, 12, 1), (228, 16, 0), (228, 24, 1),
    (260, 64, 0), (304, 64, 0), (320, 12, 1), (360, 12, 0), (360, 16, 1), (400, 64, 0), (500, 16, 1), (640, 64, 0)])
def test_k_ranges_in_parts_where_they_pay(lib, items, steps, balanced):
    """One token row to a group: as many work items as groups times weight tiles, on 152 SMs."""
    assert tile_of(lib, [1] * 4, items // 4 * 128, steps * 256, False) == (16, balanced)
