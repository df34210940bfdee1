"""The rules by which csrc/mx_gemm.hip chooses a tile of the MXFP4 products, for tests that name the
tile that they are about."""


def _sizes(R, E):
    experts = min(E, R)
    m = -(-R // experts)
    return experts, m


def forward_tile(R, E, N, Kd):
    """(rows, columns) of a tile of pmoe_mx_grouped_gemm; 256 or 192 rows: the persistent kernel."""
    experts, m = _sizes(R, E)
    items = lambda bm, bn: experts * -(-m // bm) * -(-N // bn)
    wide, least = (192, 512) if Kd % 128 else (256, 160)
    if m > 112 and items(wide, 256) >= least:
        return wide, 256
    if m > 8 and items(128, 256) >= 128:
        return 128, 256
    if m > 8 and items(128, 128) >= 128:
        return 128, 128
    return (32, 128) if items(32, 128) >= 256 else (32, 64)


def backward_tile(R, E, N, Kd):
    """(rows, columns) of a tile of pmoe_mx_grouped_gemm_backward."""
    experts, m = _sizes(R, E)
    items = lambda bm, bk: experts * -(-m // bm) * -(-Kd // bk)
    if m > 24 and items(128, 512) >= 200:
        return 128, 512
    if m > 24 and items(64, 256) >= 256:
        return 64, 256
    return (32, 512) if items(32, 512) >= 256 else (32, 128)


def persistent_tiles(offsets, N, Kd):
    """How many tiles the persistent kernel has in all; its 256 workgroups share them."""
    rows = 192 if Kd % 128 else 256
    return sum(-(-(int(b) - int(a)) // rows) for a, b in zip(offsets[:-1], offsets[1:])) * -(-N // 256)
