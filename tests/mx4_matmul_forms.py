"""Sizes of products of 4-bit tokens for every kernel form that the library builds: whether the kernel
rounds the tokens itself, T, N, K, and the form that the sizes select (the numbers of Mx4MatmulForm in
csrc/mx4_matmul_form.hpp).  Each has remainders in T, N and K; some sizes of a form fill more than one
workgroup or wave with blocks, some less than one.  Test code only."""

FORMS = [
    (True, 5, 9, 2139, 0), (True, 13, 1001, 333, 0),
    (True, 5, 8201, 2139, 1), (True, 15, 16357, 601, 1),
    (True, 5, 16377, 1115, 2), (True, 11, 40001, 271, 2),
    (False, 5, 9, 2139, 0), (False, 13, 16377, 1115, 0),
    (False, 5, 65531, 1115, 1), (False, 15, 70003, 71, 1),
    (False, 29, 9, 2139, 3), (False, 19, 4071, 1115, 3),
    (False, 29, 4105, 2139, 4), (False, 61, 2057, 1115, 4),
    (False, 61, 8201, 2139, 5), (False, 131, 2057, 9243, 5), (False, 205, 33, 4571, 5),
    (False, 301, 8201, 601, 6), (False, 1003, 4569, 2139, 6),
    (False, 61, 100003, 271, 7), (False, 301, 16393, 1115, 7),
    (False, 1501, 5333, 2139, 8), (False, 2051, 8201, 4571, 8),
    (False, 1999, 8151, 1115, 9), (False, 3001, 4569, 2139, 9),
]
