"""The library's own choice of kernel for a linear-layer product, asked on the host, so that a
test can hold that its sizes reach the kernel it is about."""
import ctypes

from fp64_gemm_emulation_amd import binding as oz

# the tiles of csrc/oz2_linear.hpp, in its order
TILES = ("tile256", "tile128", "tile64", "few8", "few16", "tile128deep")


class _Plan(ctypes.Structure):
    _fields_ = [("tile", ctypes.c_int), ("splits", ctypes.c_int)]

    def named(self):
        return TILES[self.tile], self.splits


# oz2::plan_product and oz2::plan_pair
_product = oz._LIB._ZN3oz212plan_productEblllbb
_product.restype, _product.argtypes = _Plan, [ctypes.c_bool, *[ctypes.c_long] * 3, ctypes.c_bool, ctypes.c_bool]
_pair = oz._LIB._ZN3oz29plan_pairElllRNS_4PlanES1_
_pair.restype, _pair.argtypes = ctypes.c_bool, [*[ctypes.c_long] * 3, *[ctypes.POINTER(_Plan)] * 2]


def forward(p, q, r):
    """(tile, parts of the depth) of ozaki2_linear."""
    return _product(False, p, r, q, False, False).named()


def int8(p, q, r):
    """The same of ozaki2_linear_i8."""
    return _product(True, p, r, q, False, False).named()


def backward(p, q, r):
    """(one launch for both, dX's plan, dW's plan) of ozaki2_linear_bwd."""
    dx, dw = _Plan(), _Plan()
    paired = _pair(p, q, r, ctypes.byref(dx), ctypes.byref(dw))
    return paired, dx.named(), dw.named()


# Sizes (p, q, r) that reach every kernel: one, two and more stages of the depth (64 elements of
# 16 bits, 128 of 8), whole and cut ones; rows, columns and depths that end inside a tile, a
# vector and a fragment.  With each the kernel, and whether the depth is split and joined.
FORWARD = [
    ((3900, 40, 4000), "tile256", False), ((3901, 128, 4003), "tile256", False), ((3900, 200, 4000), "tile256", False),
    ((3901, 331, 4003), "tile256", False), ((3000, 136, 2500), "tile128", False), ((3001, 331, 2499), "tile128", False),
    ((5567, 1959, 8), "tile128", True), ((1000, 256, 2048), "tile128deep", False), ((999, 331, 2047), "tile128deep", False),
    ((86, 592, 41), "tile128deep", True), ((40, 200, 1000), "tile64", False), ((33, 2048, 130), "tile64", True),
    ((37, 4099, 515), "tile64", True), ((7, 1000, 515), "few8", False), ((13, 1000, 515), "few16", False),
]
INT8 = [
    ((3900, 80, 4000), "tile256", False), ((3901, 256, 4003), "tile256", False), ((3900, 661, 4000), "tile256", False),
    ((3000, 336, 2500), "tile128", False), ((6397, 3722, 9), "tile128", True), ((203, 700, 2047), "tile128deep", False),
    ((67, 1302, 9), "tile128deep", True), ((40, 200, 1000), "tile64", False), ((33, 2048, 130), "tile64", True),
    ((1, 1000, 4099), "few16", False), ((2, 1000, 4100), "few16", False), ((2, 1003, 515), "few8", False),
    ((5, 1003, 515), "few8", False), ((13, 1003, 515), "few16", False),
]
# (p, q, r), both in one launch, dX's kernel and split, dW's
BACKWARD = [
    ((3900, 4000, 200), False, ("tile256", False), ("tile128deep", True)),
    ((3901, 4003, 203), False, ("tile256", False), ("tile128deep", True)),
    ((200, 4000, 3900), False, ("tile128deep", True), ("tile256", False)),
    ((203, 4003, 3901), False, ("tile128deep", True), ("tile256", False)),
    ((1600, 4000, 3900), False, ("tile128", False), ("tile256", False)),
    ((320, 2056, 4100), False, ("tile128deep", True), ("tile128", False)),
    ((130, 2778, 7486), False, ("tile128", True), ("tile128", False)),
    ((1601, 5808, 9), False, ("tile128", False), ("tile128", True)),
    ((50, 2048, 4096), False, ("tile64", True), ("tile128", False)),
    ((1, 8328, 810), False, ("tile64", False), ("tile128", False)),
    ((81, 8733, 823), False, ("tile128deep", False), ("tile128", False)),
    ((776, 8961, 30), False, ("tile128", False), ("tile128deep", False)),
    ((256, 256, 1024), True, ("tile128deep", True), ("tile128deep", False)),
    ((478, 8, 8), True, ("tile128deep", False), ("tile128deep", True)),
    ((1001, 999, 1003), True, ("tile128deep", False), ("tile128deep", False)),
]


def kernel(plan):
    """(tile, whether the depth is split) of a plan."""
    return plan[0], plan[1] > 1
