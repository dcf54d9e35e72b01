"""Sizes that together run every compiled form of the MX4 products and of the experts' kernels (test_mx4_plans.py
holds them to it), and GPU data whose sums are exact in fp32, so that results compare bit for bit."""
import torch

from decode_gemv_thinkbit_amd import qlinear as ql

# (M, N, K): one to four tiles of 16 rows a workgroup, whole and partial pairs of chunks, K whole and split
GEMV = ([(M, N, K) for M in (2, 3, 7, 16) for N, K in ((33, 512), (63, 736), (4100, 256), (4099, 288), (12301, 256),
                                                       (12300, 288))]
        + [(1, 5, 16384), (2, 3, 17440), (4, 2, 16384), (3, 1, 17440), (8, 17, 12288), (5, 7, 12320), (16, 4, 8192),
           (9, 6, 8224), (2, 1000, 28672), (2, 1050, 28704), (3, 1000, 16384), (4, 1001, 17440), (8, 1000, 12288),
           (6, 1003, 12320), (16, 1000, 12288), (11, 999, 12320), (2, 2000, 28672), (1, 4100, 17440), (3, 2000, 16384),
           (4, 2001, 17440), (8, 2053, 12288), (7, 2052, 12320), (16, 2000, 12288), (13, 1999, 12320)])
GEMM = ([(M, N, K) for M in (9, 20, 50) for N, K in ((33, 512), (63, 736), (4100, 256), (4099, 288), (8201, 256),
                                                     (8200, 288))]
        + [(16, 3, 16384), (9, 5, 17440), (32, 9, 12288), (20, 4, 12320), (64, 6, 8192), (50, 7, 8224), (9, 1000, 16384),
           (12, 1001, 17440), (20, 1000, 12288), (17, 999, 12320), (50, 1000, 12288), (33, 1002, 12320), (9, 2000, 16384),
           (16, 2001, 17440), (20, 2053, 12288), (32, 2052, 12320), (50, 2000, 12288), (64, 1999, 12320)]
        # output tiles of 64 x 64, 64 x 128, 128 x 128 and 256 x 256; 0 to 3 chunks past whole quads, whole quads alone
        + [(M, N, K) for M, N in ((77, 130), (140, 16390), (120, 16500), (140, 50100), (500, 12000), (700, 13001))
           for K in (128, 256, 288, 512, 736, 1056, 2080, 2176)])

# (T, k, E, H, I)
MOE = [(1, 1, 3, 32, 32), (1, 3, 5, 256, 512), (1, 8, 20, 288, 96), (1, 5, 7, 96, 1056), (1, 16, 16, 256, 1280),
       (1, 16, 17, 96, 1120), (1, 12, 40, 512, 256),
       (2, 1, 4, 256, 256), (2, 2, 6, 96, 160), (2, 16, 16, 256, 1280), (2, 8, 16, 96, 2080),
       (2, 3, 3, 64, 12288), (2, 3, 3, 96, 12320), (2, 3, 3, 256, 6144), (2, 3, 3, 96, 6176), (2, 2, 8, 256, 2048),
       (2, 2, 8, 288, 2080), (3, 3, 4, 64, 4096), (3, 3, 4, 96, 4128), (2, 2, 2, 512, 3328), (2, 2, 2, 96, 3360),
       (4, 2, 8, 256, 768), (5, 2, 10, 256, 1600), (5, 2, 10, 96, 1568), (3, 8, 64, 512, 224),
       (8, 8, 64, 256, 512), (8, 8, 64, 224, 288), (32, 2, 2, 256, 256), (40, 1, 1, 96, 288),
       (16, 4, 4, 512, 256), (17, 4, 9, 288, 96),                              # many tasks, few waves
       (9, 8, 60, 256, 1024), (9, 8, 60, 96, 1024), (16, 8, 128, 64, 928),     # many waves of the first kernel
       (9, 8, 60, 2048, 256), (9, 8, 60, 2016, 96),                            # of the second
       (64, 16, 130, 1536, 256), (64, 16, 130, 1568, 96)]                      # 64 rows a task in the second

HALVES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def mx4(codes, scales):
    """Mx4Tensor of whole codes (0..15 an element) and scale bytes, GPU tensors."""
    return ql.Mx4Tensor((codes[..., 0::2] | codes[..., 1::2] << 4).contiguous(), scales.contiguous())


def values(t):
    """fp64 values of an Mx4Tensor, by table, on its device."""
    c = torch.stack((t.codes & 15, t.codes >> 4), -1).flatten(-2).long()
    table = torch.tensor(HALVES + tuple(-v for v in HALVES), dtype=torch.float64, device=c.device)
    s = t.scales[..., :c.shape[-1] // 32].repeat_interleave(32, -1).double()
    return table[c] * torch.exp2(s - 127)


def integers(rows, K, g, dev):
    """A random matrix of every code, scales 1/2, 1 and 2: multiples of 1/4 up to 12."""
    return mx4(torch.randint(0, 16, (*rows, K), generator=g, device=dev, dtype=torch.uint8),
               torch.randint(126, 129, (*rows, 4 * ((K + 127) // 128)), generator=g, device=dev, dtype=torch.uint8))


def exact_product(x, w, unit):
    """x w^T in fp64 for values that are multiples of `unit` once multiplied: every partial sum, in any order, is
    below 2^24 units and so exact in fp32."""
    wt = w.t().contiguous()
    assert float((x.abs() @ wt.abs()).max()) < 2 ** 24 * unit
    return x @ wt
