"""Sizes of layer norm gradients for every form that the kernel takes: many rows, whose columns the row groups
sum in registers (up to 16384 columns) or other workgroups in parts, few rows, and their length.  Each length
has a remainder in 8 and lanes without a vector, but for those at the end.  Test code only."""

# (many rows, few rows, d)
SIZES = [
    (20011, 5, 101), (9001, 7, 203), (5003, 9, 301),        # 16, 32 and 64 lanes a row
    (5003, 11, 1003), (3001, 6, 1501), (2603, 5, 2001),     # 2 to 16 waves, whole rows of them as make 8
    (2201, 4, 2403), (1801, 5, 3055), (1301, 4, 3501), (1301, 5, 4091), (1103, 3, 4603), (1031, 3, 5101),
    (1031, 4, 5611), (1029, 3, 6101), (1028, 3, 6603), (1027, 5, 7001), (1027, 3, 7605), (1029, 2, 8101),
    (1031, 7, 8203), (1026, 9, 12001),                      # two vectors a lane
    (1100, 5, 20001), (1030, 3, 30001),                     # three and four
    (5003, 12, 512), (1300, 12, 4096), (1031, 12, 8192),    # no remainder, no lane without a vector
]
